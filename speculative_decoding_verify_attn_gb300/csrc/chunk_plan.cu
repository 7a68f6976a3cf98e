// What surrounds the chunk kernels (chunk_tc.cu, chunk_f32.cu): the plan that cuts a ragged batch
// into pieces of work, the append of new K/V rows to their pages, and the merge of split tiles.
//
// A row tile (row_tile consecutive rows of one sequence's chunk, for one kv head) needs the key units
// its rows see; under the causal mask these differ from tile to tile, and lengths are known on the
// device only.  One CTA therefore plans each call: with U units in all, a tile of more than
// per = ceil(U / grid) units is cut into equal pieces of at most `per`, and the pieces are sorted by
// size in descending order (a counting sort over 256 sizes), so that CTA c taking pieces c,
// 2 grid - 1 - c, 2 grid + c, ... gets nearly equal work.  The order among equal sizes varies from
// run to run; it decides only who computes a piece, and pieces are merged in key order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 256;
constexpr int kPlanMaxB = 4096;

__device__ __forceinline__ int chunk_tiles(const ServeAttnParams& p, const SeqInfo& s) {
  return s.len > 0 ? (int)(((int64_t)s.n * p.G + p.row_tile - 1) / p.row_tile) : 0;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan(const __grid_constant__ ServeAttnParams p) {
  pdl_launch_dependents();
  __shared__ int s_pre[kPlanMaxB + 1];  // tiles of the sequences before b
  __shared__ int64_t s_warp[32];
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
  __syncthreads();

  // ---- tiles per sequence, and their prefix
  int64_t run = 0;
  for (int b0 = 0; b0 < p.B && run <= p.max_tiles; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.B) {
      const SeqInfo s = seq_info(p, b);
      n = chunk_tiles(p, s);
      if (s.bad) status_report(p.status, s.bad);
    }
    int64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int64_t pre = run, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) pre += s_warp[w];
      all += s_warp[w];
    }
    if (b < p.B) s_pre[b] = (int)min(pre + x - n, (int64_t)p.max_tiles);
    run += all;
    __syncthreads();
  }
  // ranges that overlap can add up to more rows than there are: the plan then has no room for them
  const int tiles = run <= p.max_tiles ? (int)run : 0;
  if (tid == 0) {
    s_pre[p.B] = tiles;
    if (tiles != run) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_RANGE);
  }
  __syncthreads();

  struct Tile {
    int b, row0, u0, u1;
  };
  auto tile_of = [&](int t) {
    int lo = 0, hi = p.B;  // the last b with s_pre[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= t) lo = mid;
      else hi = mid;
    }
    Tile r;
    r.b = lo;
    const SeqInfo s = seq_info(p, lo);
    r.row0 = (t - s_pre[lo]) * p.row_tile;
    const int last = min(s.n * p.G, r.row0 + p.row_tile) - 1;
    const int base = s.len - s.n;
    const int first_key = p.window > 0 ? max(0, base + r.row0 / p.G + 1 - min(p.window, s.len)) : 0;
    r.u0 = first_key / p.unit_keys;
    r.u1 = (base + last / p.G) / p.unit_keys + 1;
    return r;
  };

  // ---- total units
  int64_t mine = 0;
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const Tile r = tile_of(t);
    mine += r.u1 - r.u0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) total += s_sum[w];
  const int per = (int)max((int64_t)1, (total * p.Hkv + p.grid - 1) / p.grid);

  // pieces of a tile and the bin of their size; a tile is left whole where the records would not
  // hold its pieces (sum of ceil(n / per) over tiles of n > per units is below 2 grid / Hkv)
  auto pieces_of = [&](int n) { return n > per ? (n + per - 1) / per : 1; };
  auto bin_of = [&](int n, int k) {
    const int size = (n + k - 1) / k;
    return kPlanBins - 1 - (int)((int64_t)size * (kPlanBins - 1) / per);
  };
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const Tile r = tile_of(t);
    const int n = r.u1 - r.u0, k = pieces_of(n);
    atomicAdd(&s_bin[bin_of(n, k)], k);
  }
  __syncthreads();
  if (warp == 0) {  // exclusive prefix of the bins
    int carry = 0;
    for (int i0 = 0; i0 < kPlanBins; i0 += 32) {
      const int n = s_bin[i0 + lane];
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      s_bin[i0 + lane] = carry + x - n;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      p.plan->n_items = carry;
    }
  }
  __syncthreads();
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const Tile r = tile_of(t);
    const int n = r.u1 - r.u0, k = pieces_of(n);
    const int at = atomicAdd(&s_bin[bin_of(n, k)], k);
    int slot = -1;
    if (k > 1) {
      slot = atomicAdd(&s_slots, k);
      p.splits[atomicAdd(&s_splits, 1)] = ChunkSplit{r.b, r.row0, slot, k};
    }
    for (int i = 0; i < k; ++i) {
      ChunkItem it;
      it.b = r.b;
      it.row0 = r.row0;
      it.u0 = r.u0 + (int)((int64_t)n * i / k);
      it.u1 = r.u0 + (int)((int64_t)n * (i + 1) / k);
      it.slot = k > 1 ? slot + i : -1;
      it.pad0 = it.pad1 = it.pad2 = 0;
      p.items[at + i] = it;
    }
  }
  __syncthreads();
  if (tid == 0) p.plan->n_splits = s_splits;
}

// Sequence blockIdx.x's new K and V rows, a thread per 16-byte chunk.
__global__ void __launch_bounds__(256) chunk_append(const __grid_constant__ ServeAttnParams p, int elem) {
  pdl_launch_dependents();
  const int b = blockIdx.x, per_row = p.D * elem / 16;
  const SeqInfo s = seq_info(p, b);
  const int64_t total = s.len > 0 ? (int64_t)s.n * p.Hkv * per_row : 0;
  pdl_wait();  // the plan clears the status word first
  for (int64_t i = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.y * blockDim.x) {
    const int c = (int)(i % per_row);
    const int g = (int)(i / per_row % p.Hkv);
    const int j = (int)(i / per_row / p.Hkv);
    const int64_t to = key_offset(p, s, b, g, s.len - s.n + j);
    if (to < 0) {
      atomicOr(p.status, (uint32_t)SPEC_STATUS_BAD_PAGE);
      continue;
    }
    const int64_t from = (int64_t)(s.q0 + j) * p.new_st + (int64_t)g * p.new_sh;
    const char *kn = reinterpret_cast<const char*>(p.k_new), *vn = reinterpret_cast<const char*>(p.v_new);
    char *kc = reinterpret_cast<char*>(p.k), *vc = reinterpret_cast<char*>(p.v);
    *reinterpret_cast<uint4*>(kc + to * elem + c * 16) = __ldg(reinterpret_cast<const uint4*>(kn + from * elem + c * 16));
    *reinterpret_cast<uint4*>(vc + to * elem + c * 16) = __ldg(reinterpret_cast<const uint4*>(vn + from * elem + c * 16));
  }
}

// Merge of split tiles, thread m a row, 8 columns per CTA; records are column-major, so a warp's
// loads of one column are one line.  Also zeros the rows of sequences with a bad kv_len.
constexpr int kChunkMergeCols = 8;
__global__ void __launch_bounds__(128) chunk_merge(const __grid_constant__ ServeAttnParams p) {
  pdl_wait();
  const int flat = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  for (int b = flat; b < p.B; b += gridDim.x * gridDim.y * gridDim.z) {
    const SeqInfo s = seq_info(p, b);
    if (s.len > 0 || s.n == 0) continue;
    for (int64_t i = threadIdx.x; i < (int64_t)s.n * p.Hq * p.D; i += blockDim.x) {
      const int64_t r = i / p.D;
      const int64_t off = (s.q0 + r / p.Hq) * p.o_st + (r % p.Hq) * p.o_sh + i % p.D;
      if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[off] = __float2bfloat16_rn(0.f);
      else reinterpret_cast<float*>(p.o)[off] = 0.f;
    }
  }
  const int n_splits = __ldcg(&p.plan->n_splits);
  const int d0 = blockIdx.z * kChunkMergeCols;
  for (int x = blockIdx.x; x < n_splits * p.Hkv; x += gridDim.x) {
    const int g = x % p.Hkv;
    const int4 sp = __ldcg(reinterpret_cast<const int4*>(p.splits + x / p.Hkv));
    const ChunkSplit split{sp.x, sp.y, sp.z, sp.w};
    const SeqInfo s = seq_info(p, split.b);
    const int m = blockIdx.y * blockDim.x + threadIdx.x;
    if (m >= p.row_tile || split.row0 + m >= s.n * p.G) continue;
    float M = neg_inf();
    for (int i = 0; i < split.pieces; ++i)
      M = fmaxf(M, __ldcg(&p.part_ml[((int64_t)(split.slot + i) * p.Hkv + g) * p.row_tile + m]).x);
    float L = 0.f, acc[kChunkMergeCols];
#pragma unroll
    for (int e = 0; e < kChunkMergeCols; ++e) acc[e] = 0.f;
    if (M != neg_inf()) {
#pragma unroll 2
      for (int i = 0; i < split.pieces; ++i) {
        const int64_t rec = (int64_t)(split.slot + i) * p.Hkv + g;
        const float2 ml = __ldcg(&p.part_ml[rec * p.row_tile + m]);
        const float w = ml.x == neg_inf() ? 0.f : exp2f(ml.x - M);
        const float* src = p.part_o + (rec * p.D + d0) * p.row_tile + m;
        L += w * ml.y;
#pragma unroll
        for (int e = 0; e < kChunkMergeCols; ++e) {
          // a piece in which the row saw nothing holds no value
          const float v = __ldcg(src + e * p.row_tile);
          acc[e] = fmaf(w, ml.x == neg_inf() ? 0.f : v, acc[e]);
        }
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const int64_t off = o_offset(p, s, g, split.row0 + m) + d0;
    if (p.o_bf16) {
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + off;
      if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
        uint4 v;
        v.x = pack_bf16(acc[0] * inv, acc[1] * inv);
        v.y = pack_bf16(acc[2] * inv, acc[3] * inv);
        v.z = pack_bf16(acc[4] * inv, acc[5] * inv);
        v.w = pack_bf16(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(dst) = v;
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

cudaError_t launch_chunk_plan(const ServeAttnParams& p, cudaStream_t stream) {
  chunk_plan<<<1, kPlanThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_chunk_append(const ServeAttnParams& p, int elem_bytes, cudaStream_t stream) {
  const int64_t want = ((int64_t)p.max_q * p.Hkv * (p.D * elem_bytes / 16) + 255) / 256;
  const int64_t most = p.B < 4096 ? 4096 / p.B : 1;  // about 4096 CTAs of 256 threads at most
  return launch_dependent(chunk_append, dim3(p.B, (unsigned)(want < most ? want : most)), dim3(256), 0, stream, 0u, p,
                          elem_bytes);
}
cudaError_t launch_chunk_merge(const ServeAttnParams& p, cudaStream_t stream) {
  const unsigned threads = p.row_tile < 128 ? p.row_tile : 128;
  const dim3 grid(p.grid, p.row_tile / threads, p.D / kChunkMergeCols);
  return launch_dependent(chunk_merge, grid, dim3(threads), 0, stream, 0u, p);
}

}  // namespace specv
