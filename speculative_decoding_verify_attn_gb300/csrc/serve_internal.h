// Internal interface between serve_api.cpp and the kernels of the serving operators (paged_mma.cu,
// chunk_tc.cu, chunk_f32.cu, logprobs.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace specv {

// CTAs a chunk kernel's work is split over at most (one per SM); the workspace is sized for it.
constexpr int kServeMaxGrid = 160;
// Query rows (tokens x heads of a group) per sequence and kv head up to which the mma.sync kernel
// runs.
constexpr int kMmaMaxRows = 32;
constexpr int kMmaUnit = 128;   // keys per unit of work of the mma.sync kernel (16 per warp)
// The same over 8-bit caches: keys of a unit that a warp takes, warps of a CTA for rows of 128 and of 64.
constexpr int kMma8Keys = 32;
constexpr int kMma8Warps = 8;
constexpr int kMma8WideWarps = 12;
// Segments of at most this many keys are one CTA of the mma.sync kernel each (no merge launch).  Device
// time with and without: 8 segments of 128 keys 5.2 and 6.9 us, 256 segments of 512 keys 15.4 and 17.5;
// past it 8 segments of 1024 keys take 11.3 and 8.4.
constexpr int kMmaDirectKeys = 4 * kMmaUnit;
constexpr int kTcRows = 256;    // query rows per tile of the tcgen05 kernel (two blocks of 128)
constexpr int kTcKeys = 128;    // keys per unit of work of the tcgen05 kernel
// Tokens per page from which the tcgen05 kernel copies pages by TMA, below cp.async.  A 2048-token chunk at
// 32K by TMA and by cp.async: pages of 16 961 and 753 us, of 32 763 and 722, of 64 674 and 706.
constexpr int kTmaMinPage = 64;
constexpr int kF32Rows = 64;    // query rows per tile of the fp32 kernel
constexpr int kF32Keys = 64;    // keys per unit of work of the fp32 kernel

// One piece of work of a chunk kernel: the row tile starting at row `row0` of sequence b (row r: token
// r / G of the chunk, head r % G of the group) of kv head g (small tiles: of every kv head), key units
// [u0, u1).  slot < 0: the piece is the whole tile and writes o; else its record.  The sequence's own
// numbers (serve_common.cuh) come along, so that a piece costs its reader one trip to memory.
struct alignas(16) ChunkItem {
  int32_t b, row0, u0, u1, slot, q0, n, len, lo, g, pad0, pad1;
};
// A tile cut over CTAs c0 .. c1: its first record is 2 c0 + first, the others 2 c.
struct alignas(16) ChunkSplit {
  int32_t b, row0, g, c0, c1, first, pad0, pad1;
};
// Head of the plan in the workspace, after the status block (see chunk_plan.cu).
struct ChunkPlan {
  int32_t n_small, n_splits, big_ctas, small_first;
};
// Tiles of more than a quarter of a CTA's share are cut; such a share holds eight pieces at most.
constexpr int kBigFraction = 4;
constexpr int kBigPieces = 8;
constexpr int kMaxBig = kBigFraction * kServeMaxGrid;

// Light calls: no tile has more than this many units and the batch this many sequences at most, so tiles
// are not cut, and every CTA works its tiles out by itself: no plan, no merge launch.  Planned and light:
// 32 chunks over a window of 512 26 and 20 us of device time (with append 26 and 22), a 16K prompt with
// that window 190 and 173 us.
constexpr int kLightUnits = 8;
constexpr int kLightMaxB = 64;

struct ServeAttnParams {
  int B, Hq, Hkv, G, D, T, max_q, window;
  int paged, page_size, num_pages, table_cols;
  int page_shift;         // log2(page_size), or -1
  const int32_t* table;
  int64_t table_stride;
  const int32_t* q_start;
  const int32_t* kv_len;  // null for packed prompts: the length is the chunk's own
  const void* q;
  int64_t q_st, q_sh;
  void* k;                // pages, or the packed rows
  void* v;
  int64_t kv_sp, kv_sh, kv_st;
  const void* k_new;
  const void* v_new;
  int64_t new_st, new_sh;
  void* o;
  int64_t o_st, o_sh;
  int o_bf16;
  float scale_log2;       // scale * log2(e)
  int grid;               // CTAs of the attention kernel
  int direct;             // mma.sync kernel: a CTA per segment, no records
  int row_tile, unit_keys;  // chunk kernels: rows per tile, keys per unit
  int light;              // chunk kernels: a light call (above)
  int first;              // chunk kernels: the attention kernel is the call's first and clears the status
  // chunk kernels: what a piece costs beside its units (its rows, its first maximum, its epilogue), and
  // what cutting costs a CTA (a second cut tile's piece, the merge), in units
  float piece_cost, cut_cost;
  int share_piece;        // chunk kernels: what a piece counts in the shares of cut tiles beside its units, in units
  int min_units;          // chunk kernels: units a CTA's share of cut tiles has at least
  int use_tma;            // tcgen05 kernel: the tensor maps are valid
  int tma_page_keys;      // keys one copy brings (min(page_size, kTcKeys); packed: kTcKeys)
  int max_tiles;          // chunk kernels: tiles (per kv head) the plan has room for
  uint32_t* status;
  ChunkPlan* plan;
  int32_t* big_count;     // [kServeMaxGrid]: pieces of cut tiles a CTA has
  ChunkItem* big;         // [kServeMaxGrid][kBigPieces]
  ChunkItem* items;       // small tiles, largest first
  ChunkSplit* splits;     // [kServeMaxGrid]
  float2* part_ml;        // chunk kernels [2 * cta + s][row_tile]; mma: [2 * cta + s][kMmaMaxRows]
  float* part_o;          // chunk kernels [2 * cta + s][D][row_tile]; mma: [..][kMmaMaxRows][D]
};

// Upper bounds on what the plan can hold.
inline int64_t chunk_max_tiles(int64_t T, int G, int B, int row_tile) { return T * G / row_tile + B; }

size_t mma_workspace_bytes(int D);
size_t chunk_workspace_bytes(int64_t T, int G, int B, int D, int row_tile);
void mma_workspace_carve(void* ws, ServeAttnParams* p);
void chunk_workspace_carve(void* ws, ServeAttnParams* p);

cudaError_t launch_paged_mma(const ServeAttnParams& p, cudaStream_t stream);
// joins the records of segments over 8-bit caches that several CTAs of `warps` warps share
cudaError_t launch_paged8_merge(const ServeAttnParams& p, int warps, cudaStream_t stream);
// plan and append, attention, merge
cudaError_t launch_chunk_prepare(const ServeAttnParams& p, int elem_bytes, cudaStream_t stream);
cudaError_t launch_chunk_tc(const ServeAttnParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                            cudaStream_t stream);
cudaError_t launch_chunk_f32(const ServeAttnParams& p, cudaStream_t stream);
cudaError_t launch_chunk_merge(const ServeAttnParams& p, cudaStream_t stream);

struct LogprobParams {
  int N, V, K, bf16, slices;
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_lp;
  uint32_t* status;
  float4* part_stat;               // [N][slices]: max, sum, weighted sum
  unsigned long long* part_keys;   // [N][slices][K]
};
int logprob_slices(int N, int V);
size_t logprob_workspace_bytes(int N, int V, int K);
void logprob_workspace_carve(void* ws, LogprobParams* p);
cudaError_t launch_token_logprobs(const LogprobParams& p, cudaStream_t stream);

}  // namespace specv
