// Internal interface between cache_api.cpp and the kernels of the cache operators (rotary.cu,
// kv8_append.cu, paged8_mma.cu, chunk8_tc.cu, pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "serve_internal.h"
#include "spec_cache.h"

namespace specv {

// ------------------------------------------------------------------ rotary positions
struct RotaryParams {
  int T, Hq, Hkv, D, rot, pairs, f32, B, negate;
  int tile;               // tokens per CTA
  float amplitude;
  const void* q;
  int64_t q_st, q_sh;
  const void* k;
  int64_t k_st, k_sh;
  void* qo;
  int64_t qo_st, qo_sh;
  void* ko;
  int64_t ko_st, ko_sh;
  int copy_q, copy_k;     // values past rot have to be copied (not in place)
  const unsigned long long* steps;
  const int32_t* positions;
  const int32_t* q_start;
  const int32_t* kv_len;
  uint32_t* status;
};
constexpr int kRotaryMaxTile = 8;
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream);

// ------------------------------------------------------------------ the cache in 8 bits
// Exponent bytes that count: 2^-64 .. 2^64.
constexpr int kMinExpByte = 63, kMaxExpByte = 191;

struct Kv8Params : ServeAttnParams {
  uint8_t* k_exp;
  uint8_t* v_exp;
  int64_t exp_sp, exp_sh;
  int block, block_shift;  // log2(block), or -1
  int src_f32;             // k_new, v_new in 32 bits
};
// `first`: the kernel is the call's first and clears the status; else it runs behind the one that does.
cudaError_t launch_kv8_append(const Kv8Params& p, bool first, cudaStream_t stream);
// p.first: the attention kernel is the call's first.
cudaError_t launch_paged8_mma(const Kv8Params& p, cudaStream_t stream);
cudaError_t launch_chunk8_tc(const Kv8Params& p, cudaStream_t stream);

// ------------------------------------------------------------------ pages
struct PageRow {  // what a row becomes
  int32_t parent, before, kept, need, last, writes, pad0, pad1;
};
struct PageParams {
  int B, cols, page_size, num_pages, compact;
  const int32_t* table;
  int64_t table_st;
  const int32_t* held;
  const int32_t* kv_len;
  const int32_t* refs;
  const int32_t* parent;
  const int32_t* grow;
  int32_t* table_out;
  int64_t table_out_st;
  int32_t* held_out;
  int32_t* kv_len_out;
  int32_t* refs_out;
  int32_t* moved_out;
  int32_t* num_live;
  // workspace
  uint32_t* status;
  int32_t* n_pairs;   // moves that the copying kernel makes
  int2* pairs;        // (from, to)
  int32_t* count;     // [num_pages] holders
  int32_t* writers;   // [num_pages] rows that write to a page they got from their parent
  int32_t* lowest;    // [num_pages] the lowest of them
  int32_t* free_ids;  // [num_pages] free pages in ascending order; compact: pages' new ids
  PageRow* rows;      // [B]
  int32_t* stage;     // [B][cols] entries of rows that change their parent
};
struct PageArrays {
  static constexpr int kMax = 48;
  int n;
  int32_t pieces[kMax + 1];  // pieces of 16 KB of a page before each array
  char* base[kMax];
  int64_t stride[kMax], bytes[kMax];
};
constexpr int kPagePiece = 16384;
size_t page_workspace_bytes(int B, int cols, int num_pages, bool compact);
void page_workspace_carve(void* ws, PageParams* p);
cudaError_t launch_page_fork(const PageParams& p, cudaStream_t stream);
cudaError_t launch_page_compact(const PageParams& p, cudaStream_t stream);
cudaError_t launch_page_copy(const PageParams& p, const PageArrays& a, int max_pairs, cudaStream_t stream);

}  // namespace specv
