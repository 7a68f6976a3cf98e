// What surrounds the chunk kernels (chunk_tc.cu, chunk_f32.cu): the plan that cuts a ragged batch
// into pieces of work, the append of new K/V rows to their pages, and the merge of split tiles.
//
// A row tile (row_tile consecutive rows of one sequence's chunk, for one kv head) needs the key units
// its rows see; under the causal mask these differ from tile to tile, and lengths are known on the
// device only.  One CTA therefore plans each call: with U units in all, a tile of more than
// per = ceil(U / grid) units (min_units at least) is cut into equal pieces of at most `per`, and the pieces are sorted by
// size in descending order (a counting sort over 256 sizes), so that CTA c taking pieces c,
// 2 grid - 1 - c, 2 grid + c, ... gets nearly equal work.  The order among equal sizes varies from
// run to run; it decides only who computes a piece, and pieces are merged in key order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_cache.h"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 256;

__device__ __forceinline__ int chunk_tiles(const ServeAttnParams& p, const SeqInfo& s) {
  return s.len > 0 ? (int)(((int64_t)s.n * p.G + p.row_tile - 1) / p.row_tile) : 0;
}

struct PlanTile {
  int b, row0, u0, u1;
};

__device__ __forceinline__ void plan_body(const ServeAttnParams& p, int* s_pre, int* s_n, int* s_len) {
  __shared__ uint32_t s_warp[32];
  __shared__ int64_t s_sum[32];
  __shared__ int s_bin[kPlanBins];
  __shared__ int s_slots, s_splits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    status_clear_for_launch(p.status);
    s_slots = 0;
    s_splits = 0;
  }
  if (tid < kPlanBins) s_bin[tid] = 0;

  // ---- tiles per sequence, and their prefix s_pre.  Overlapping ranges can add up to more rows than
  // there are; sums are capped where the plan has no room for them anyway.
  constexpr uint32_t kCap = 1u << 25;  // above any max_tiles
  uint32_t run = 0;
  for (int b0 = 0; b0 < p.B && run <= (uint32_t)p.max_tiles; b0 += kPlanThreads) {
    const int b = b0 + tid;
    uint32_t n = 0;
    if (b < p.B) {
      const SeqInfo s = seq_info(p, b);
      n = (uint32_t)chunk_tiles(p, s);
      s_n[b] = s.n;
      s_len[b] = s.len;
      if (s.bad) status_report(p.status, s.bad);
    }
    uint32_t x = n;  // at most 2^22 each
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = min(x, kCap);
    __syncthreads();
    const uint32_t sums = s_warp[lane];
    const uint32_t pre = run + __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u);
    run = min(run + __reduce_add_sync(0xffffffffu, sums), kCap);
    if (b < p.B) s_pre[b] = (int)min(pre + x - n, kCap);
    __syncthreads();
  }
  const int tiles = run <= (uint32_t)p.max_tiles ? (int)run : 0;
  if (tid == 0) {
    s_pre[p.B] = tiles;
    if (tiles == 0 && run > 0) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_RANGE);
  }
  __syncthreads();

  auto tile_of = [&](int t) {
    int lo = 0, hi = p.B;  // the last b with s_pre[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= t) lo = mid;
      else hi = mid;
    }
    PlanTile r;
    r.b = lo;
    const int n = s_n[lo], len = s_len[lo], base = len - n;
    r.row0 = (t - s_pre[lo]) * p.row_tile;
    const int last = min(n * p.G, r.row0 + p.row_tile) - 1;
    const int first_key = p.window > 0 ? max(0, base + r.row0 / p.G + 1 - min(p.window, len)) : 0;
    r.u0 = first_key / p.unit_keys;
    r.u1 = (base + last / p.G) / p.unit_keys + 1;
    return r;
  };
  // the usual plan has a tile per thread at most
  PlanTile own{0, 0, 0, 0};
  if (tid < tiles) own = tile_of(tid);
  auto tile = [&](int t) { return t == tid ? own : tile_of(t); };

  // ---- total units
  int64_t mine = 0;
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const PlanTile r = tile(t);
    mine += r.u1 - r.u0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  int64_t total = s_sum[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int per = (int)max((int64_t)p.min_units, (total * p.Hkv + p.grid - 1) / p.grid);

  // the sum of ceil(n / per) over tiles of n > per units is below 2 grid / Hkv, what the records hold
  auto pieces_of = [&](int n) { return n > per ? (n + per - 1) / per : 1; };
  const float bin_scale = (float)(kPlanBins - 1) / (float)per;
  auto bin_of = [&](int n, int k) {
    const int size = k == 1 ? n : (n + k - 1) / k;
    return kPlanBins - 1 - min(kPlanBins - 1, (int)((float)size * bin_scale));
  };
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const PlanTile r = tile(t);
    const int n = r.u1 - r.u0, k = pieces_of(n);
    atomicAdd(&s_bin[bin_of(n, k)], k);
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefix of the bins, 8 per lane
    int v[kPlanBins / 32], sum = 0;
#pragma unroll
    for (int i = 0; i < kPlanBins / 32; ++i) {
      v[i] = s_bin[lane * (kPlanBins / 32) + i];
      sum += v[i];
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int at = x - sum;
#pragma unroll
    for (int i = 0; i < kPlanBins / 32; ++i) {
      s_bin[lane * (kPlanBins / 32) + i] = at;
      at += v[i];
    }
    if (lane == 31) p.plan->n_items = x;
  }
  __syncthreads();
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const PlanTile r = tile(t);
    const int n = r.u1 - r.u0, k = pieces_of(n);
    const int at = atomicAdd(&s_bin[bin_of(n, k)], k);
    int slot = -1;
    if (k > 1) {
      slot = atomicAdd(&s_slots, k);
      p.splits[atomicAdd(&s_splits, 1)] = ChunkSplit{r.b, r.row0, slot, k};
    }
    const SeqInfo s = seq_info(p, r.b);
    for (int i = 0; i < k; ++i) {
      int4* dst = reinterpret_cast<int4*>(p.items + at + i);
      const int u0 = r.u0 + (k == 1 ? 0 : (int)((int64_t)n * i / k));
      const int u1 = r.u0 + (k == 1 ? n : (int)((int64_t)n * (i + 1) / k));
      dst[0] = make_int4(r.b, r.row0, u0, u1);
      dst[1] = make_int4(k > 1 ? slot + i : -1, s.q0, s.n, s.len);
      dst[2] = make_int4(s.lo, 0, 0, 0);
    }
  }
  __syncthreads();
  if (tid == 0) p.plan->n_splits = s_splits;
}

// CTA 0 makes the plan; the others (if there are new rows) append: CTA 1 + b + B y takes sequence b, a
// thread per 16-byte chunk of a row.
__global__ void __launch_bounds__(kPlanThreads) chunk_prepare(const __grid_constant__ ServeAttnParams p, int elem) {
  pdl_launch_dependents();
  extern __shared__ int s_seq[];  // [B + 1], [B], [B]
  if (blockIdx.x == 0) {
    plan_body(p, s_seq, s_seq + p.B + 1, s_seq + 2 * p.B + 1);
    return;
  }
  const int b = (blockIdx.x - 1) % p.B, y = (blockIdx.x - 1) / p.B, ny = (gridDim.x - 1) / p.B;
  const int per_row = p.D * elem / 16;
  const SeqInfo s = seq_info(p, b);
  const int64_t total = s.len > 0 ? (int64_t)s.n * p.Hkv * per_row : 0;
  for (int64_t i = (int64_t)y * blockDim.x + threadIdx.x; i < total; i += (int64_t)ny * blockDim.x) {
    const int c = (int)(i % per_row);
    const int64_t rest = i / per_row;
    const int g = (int)(rest % p.Hkv), j = (int)(rest / p.Hkv);
    const int64_t to = key_offset(p, s, b, g, s.len - s.n + j);
    if (to < 0) {
      status_report(p.status, (uint32_t)SPEC_STATUS_BAD_PAGE);
      continue;
    }
    const int64_t from = (int64_t)(s.q0 + j) * p.new_st + (int64_t)g * p.new_sh;
    const char *kn = reinterpret_cast<const char*>(p.k_new), *vn = reinterpret_cast<const char*>(p.v_new);
    char *kc = reinterpret_cast<char*>(p.k), *vc = reinterpret_cast<char*>(p.v);
    *reinterpret_cast<uint4*>(kc + to * elem + c * 16) = __ldg(reinterpret_cast<const uint4*>(kn + from * elem + c * 16));
    *reinterpret_cast<uint4*>(vc + to * elem + c * 16) = __ldg(reinterpret_cast<const uint4*>(vn + from * elem + c * 16));
  }
}

// Merge of split tiles: a unit of work is (split tile, kv head, block of kMergeRows rows, 8 columns),
// thread m a row; records are column-major, so a warp's loads of one column are one line.  The pieces'
// weights 2^(m_i - M) are worked out once per row and unit; loads go out several pieces at a time.
// Also zeros the rows of sequences with a bad kv_len.
constexpr int kChunkMergeCols = 8;
constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 4;
__global__ void __launch_bounds__(kMergeThreads) chunk_merge(const __grid_constant__ ServeAttnParams p) {
  const int rows_per = min(kMergeThreads, p.row_tile), groups = kMergeThreads / rows_per;
  const int m_in = threadIdx.x % rows_per, sub = threadIdx.x / rows_per;
  const int blocks = p.row_tile / rows_per, chunks = p.D / kChunkMergeCols;
  pdl_wait();
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const SeqInfo s = seq_info(p, b);
    if (s.len > 0 || s.n == 0) continue;
    for (int64_t i = threadIdx.x; i < (int64_t)s.n * p.Hq * p.D; i += blockDim.x) {
      const int64_t r = i / p.D;
      const int64_t off = (s.q0 + r / p.Hq) * p.o_st + (r % p.Hq) * p.o_sh + i % p.D;
      if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[off] = __float2bfloat16_rn(0.f);
      else reinterpret_cast<float*>(p.o)[off] = 0.f;
    }
  }
  const int total = __ldcg(&p.plan->n_splits) * p.Hkv * blocks * chunks;  // below 2^20
  for (int x = blockIdx.x * groups + sub; x < total; x += gridDim.x * groups) {
    const int d0 = x % chunks * kChunkMergeCols;
    const int m = x / chunks % blocks * rows_per + m_in;
    const int g = x / chunks / blocks % p.Hkv;
    const int4 sp = __ldcg(reinterpret_cast<const int4*>(p.splits + x / chunks / blocks / p.Hkv));
    const ChunkSplit split{sp.x, sp.y, sp.z, sp.w};
    const SeqInfo s = seq_info(p, split.b);
    if (split.row0 + m >= s.n * p.G) continue;
    const float2* ml = p.part_ml + ((int64_t)split.slot * p.Hkv + g) * p.row_tile + m;
    const int64_t ml_step = (int64_t)p.Hkv * p.row_tile, o_step = ml_step * p.D;
    const float* src = p.part_o + (((int64_t)split.slot * p.Hkv + g) * p.D + d0) * p.row_tile + m;
    float M = neg_inf();
#pragma unroll 8
    for (int i = 0; i < split.pieces; ++i) M = fmaxf(M, __ldcg(ml + i * ml_step).x);
    float L = 0.f, acc[kChunkMergeCols];
#pragma unroll
    for (int e = 0; e < kChunkMergeCols; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < split.pieces; i0 += kMergeBatch) {
      float2 a[kMergeBatch];
      float v[kMergeBatch][kChunkMergeCols];
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) {
        const bool in = i0 + u < split.pieces;
        a[u] = in ? __ldcg(ml + (i0 + u) * ml_step) : make_float2(neg_inf(), 0.f);
#pragma unroll
        for (int e = 0; e < kChunkMergeCols; ++e) v[u][e] = in ? __ldcg(src + (i0 + u) * o_step + e * p.row_tile) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) {
        if (a[u].x == neg_inf()) continue;  // the row saw nothing there: no value was written
        const float w = exp2f(a[u].x - M);
        L += w * a[u].y;
#pragma unroll
        for (int e = 0; e < kChunkMergeCols; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const int64_t off = o_offset(p, s, g, split.row0 + m) + d0;
    if (p.o_bf16) {
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + off;
      if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
        uint4 q;
        q.x = pack_bf16(acc[0] * inv, acc[1] * inv);
        q.y = pack_bf16(acc[2] * inv, acc[3] * inv);
        q.z = pack_bf16(acc[4] * inv, acc[5] * inv);
        q.w = pack_bf16(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(dst) = q;
      } else {
#pragma unroll
        for (int e = 0; e < kChunkMergeCols; ++e) dst[e] = __float2bfloat16_rn(acc[e] * inv);
      }
    } else {
      float* dst = reinterpret_cast<float*>(p.o) + off;
#pragma unroll
      for (int e = 0; e < kChunkMergeCols; ++e) dst[e] = acc[e] * inv;
    }
  }
}

// ------------------------------------------------------------------ workspace and launches
static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
// Records a plan can need: below 2 grid over all kv heads.
static size_t chunk_records() { return 2 * (size_t)kServeMaxGrid; }

static void chunk_layout(int64_t T, int G, int B, int D, int row_tile, size_t (&at)[6]) {
  const size_t items = (size_t)chunk_max_tiles(T, G, B, row_tile) + chunk_records();
  at[0] = 256;                                                // plan
  at[1] = at[0] + 256;                                        // items
  at[2] = up256(at[1] + items * sizeof(ChunkItem));           // splits
  at[3] = up256(at[2] + chunk_records() * sizeof(ChunkSplit));  // (m, l)
  at[4] = up256(at[3] + chunk_records() * row_tile * sizeof(float2));  // o
  at[5] = up256(at[4] + chunk_records() * row_tile * (size_t)D * sizeof(float));
}
size_t chunk_workspace_bytes(int64_t T, int G, int B, int Hkv, int D, int row_tile) {
  (void)Hkv;
  size_t at[6];
  chunk_layout(T, G, B, D, row_tile, at);
  return at[5];
}
void chunk_workspace_carve(void* ws, ServeAttnParams* p) {
  size_t at[6];
  chunk_layout(p->T, p->G, p->B, p->D, p->row_tile, at);
  char* b = reinterpret_cast<char*>(ws);
  p->status = reinterpret_cast<uint32_t*>(b);
  p->plan = reinterpret_cast<ChunkPlan*>(b + at[0]);
  p->items = reinterpret_cast<ChunkItem*>(b + at[1]);
  p->splits = reinterpret_cast<ChunkSplit*>(b + at[2]);
  p->part_ml = reinterpret_cast<float2*>(b + at[3]);
  p->part_o = reinterpret_cast<float*>(b + at[4]);
  p->max_tiles = (int)chunk_max_tiles(p->T, p->G, p->B, p->row_tile);
}

cudaError_t launch_chunk_prepare(const ServeAttnParams& p, int elem_bytes, cudaStream_t stream) {
  const int smem = (3 * p.B + 1) * (int)sizeof(int);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(chunk_prepare), smem);
  if (e != cudaSuccess) return e;
  unsigned grid = 1;
  if (p.k_new) {  // about 600 CTAs at most, one per sequence at least
    const int64_t want = ((int64_t)p.max_q * p.Hkv * (p.D * elem_bytes / 16) + kPlanThreads - 1) / kPlanThreads;
    const int64_t most = (600 + p.B - 1) / p.B;
    grid += (unsigned)p.B * (unsigned)(want < most ? want : most);
  }
  chunk_prepare<<<grid, kPlanThreads, smem, stream>>>(p, elem_bytes);
  return cudaGetLastError();
}
cudaError_t launch_chunk_merge(const ServeAttnParams& p, cudaStream_t stream) {
  return launch_dependent(chunk_merge, dim3(4 * p.grid), dim3(kMergeThreads), 0, stream, 0u, p);
}

}  // namespace specv
