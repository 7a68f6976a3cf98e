// What surrounds the chunk kernels (chunk_tc.cu, chunk_f32.cu): the plan that cuts a ragged batch
// into pieces of work, the append of new K/V rows to their pages, and the merge of split tiles.
//
// A row tile (row_tile consecutive rows of one sequence's chunk, for one kv head) needs the key units
// its rows see; under the causal mask these differ from tile to tile, and lengths are known on the
// device only.  One CTA therefore plans each call.  With U units in all a CTA's share is
// per = U / grid.  If cutting pays (see `cut` below), tiles of more than per / 4 units ("big") go to as many
// CTAs as they fill: first whole tiles, one per CTA and wave, for as many waves as leave every CTA short
// of its share; the rest is laid end to end and cut so as to fill each CTA up to its share.  Shares are thus equal to a unit,
// leave at most two records each (a cut tile at either end), and CTAs on the same keys (row tiles of
// one sequence and head) start on them together, which keeps those keys in L2: with everything cut at
// equal distances, a 2048-token chunk at 32K ran at the HBM rate of its 134 MB of keys.  The other tiles
// stay whole: sorted by size (a counting sort over 256 sizes) and dealt forth and back over the
// remaining CTAs, they differ by a fraction of a quarter share.  Big tiles keep the order of the batch,
// so a call's cuts and with them its rounding are the same every time; the order among small tiles of
// equal size varies and decides only who computes a tile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_cache.h"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

// Few threads: every instruction of the plan is paid by each of its warps, and its steps are short (four
// fp32 sequences with cut tiles: 13 800 cycles, 18 900 with 1024 threads).
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBins = 256;

struct PlanTile {
  int b, row0, u0, u1;
};

__device__ __forceinline__ void plan_body(const ServeAttnParams& p, int* s_pre, int* s_n, int* s_len, int* s_q0) {
  __shared__ uint32_t s_warp[32];
  __shared__ int64_t s_sum[32];
  __shared__ int s_bin[kPlanBins];
  __shared__ int s_big[kMaxBig];
  __shared__ int64_t s_big_at[kMaxBig + 1];
  __shared__ int64_t s_from[kServeMaxGrid];
  __shared__ int s_small, s_splits, s_waves;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    status_clear_for_launch(p.status);
    s_splits = 0;
    s_waves = kBigPieces;
  }
  for (int i = tid; i < kPlanBins; i += kPlanThreads) s_bin[i] = 0;

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
      s_q0[b] = s.q0;
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
    const uint32_t sums = lane < kPlanWarps ? s_warp[lane] : 0u;
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
    r.row0 = (t - s_pre[lo]) * p.row_tile;
    tile_units(p, s_n[lo], s_len[lo], r.row0, r.u0, r.u1);
    return r;
  };
  // the usual plan has a tile per thread at most
  PlanTile own{0, 0, 0, 0};
  if (tid < tiles) own = tile_of(tid);
  auto tile = [&](int t) { return t == tid ? own : tile_of(t); };

  // ---- total units
  int64_t mine = 0;
  uint32_t longest = 0;
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const PlanTile r = tile(t);
    mine += r.u1 - r.u0;
    longest = max(longest, (uint32_t)(r.u1 - r.u0));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) {
    s_sum[warp] = mine;
    s_warp[warp] = longest;
  }
  __syncthreads();
  int64_t total = lane < kPlanWarps ? s_sum[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  longest = __reduce_max_sync(0xffffffffu, lane < kPlanWarps ? s_warp[lane] : 0u);
  const int64_t all = total * p.Hkv;
  const int per = (int)max((int64_t)p.min_units, (all + p.grid - 1) / p.grid);
  // cut only where an estimate says that it beats dealing whole tiles, in units with piece_cost for every
  // piece: whole tiles take the longest one, or as many average ones as waves; shares take the mean, a second cut
  // tile and the merge.  The dealing leaves its longest CTA somewhat above the estimate (24 mixed sequences:
  // 134 units for an estimate of 128, and 117 on average), so batches on the border stay whole.
  const float items = (float)tiles * p.Hkv, mean = (float)all / p.grid + p.piece_cost * items / p.grid;
  const float whole_cost = fmaxf((float)longest + p.piece_cost, ceilf(items / p.grid) * (mean * p.grid / fmaxf(items, 1.f)));
  const bool cut = mean + p.cut_cost < 0.95f * whole_cost;
  auto is_big = [&](int n) { return cut && n > per / kBigFraction; };

  // ---- big tiles in the batch's order, with the units before each; small tiles by size
  const float bin_scale = (float)(kPlanBins - 1) / (cut ? (float)per / kBigFraction : (float)max(longest, 1u));
  auto bin_of = [&](int n) { return kPlanBins - 1 - min(kPlanBins - 1, (int)((float)n * bin_scale)); };
  int n_big = 0;
  int64_t big_units = 0;
  for (int t0 = 0; t0 < tiles; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int n = 0;
    if (t < tiles) {
      const PlanTile r = tile(t);
      n = r.u1 - r.u0;
    }
    const bool big = n > 0 && is_big(n);
    if (n > 0 && !big) atomicAdd(&s_bin[bin_of(n)], 1);
    const unsigned mask = __ballot_sync(0xffffffffu, big);
    int64_t x = big ? n : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();  // the sums of the round before have been read
    if (lane == 31) {
      s_warp[warp] = __popc(mask);
      s_sum[warp] = x;
    }
    __syncthreads();
    const uint32_t counts = lane < kPlanWarps ? s_warp[lane] : 0u;
    int64_t pre_units = lane < warp ? s_sum[lane] : 0, sum_units = lane < kPlanWarps ? s_sum[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      pre_units += __shfl_xor_sync(0xffffffffu, pre_units, o);
      sum_units += __shfl_xor_sync(0xffffffffu, sum_units, o);
    }
    // fewer than kMaxBig in all: each has more than a quarter of a share
    const int before = n_big + (int)__reduce_add_sync(0xffffffffu, lane < warp ? counts : 0u) + __popc(mask & ((1u << lane) - 1u));
    if (big && before < kMaxBig) {
      s_big[before] = t;
      s_big_at[before] = big_units + pre_units + x - n;
    }
    n_big += (int)__reduce_add_sync(0xffffffffu, counts);
    big_units += sum_units;
  }
  __syncthreads();
  n_big = min(n_big, kMaxBig);
  if (tid == 0) s_big_at[n_big] = big_units;
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
    if (lane == 31) s_small = x;
  }
  __syncthreads();

  // ---- shares of the big tiles: `ctas` of `share` units of the line [0, line)
  const int64_t line = big_units * p.Hkv;
  const int small = s_small;
  int ctas = 0;
  if (line > 0) {
    ctas = small == 0 ? p.grid : (int)min((int64_t)p.grid, max((int64_t)1, (line + per / 2) / per));
    ctas = (int)min((int64_t)ctas, (line + p.min_units - 1) / p.min_units);
  }
  const int64_t share = ctas > 0 ? (line + ctas - 1) / ctas : 1;
  // ---- waves of whole tiles: item i (tile i / Hkv, head i % Hkv) to CTA i % ctas
  auto big_size = [&](int j) { return (int)(s_big_at[j + 1] - s_big_at[j]); };
  const int n_items = n_big * p.Hkv;
  if (tid < ctas) {
    int64_t sum = 0;
    int k = 0;
    for (int i = tid; i < n_items; i += ctas, ++k) {
      sum += big_size(i / p.Hkv);
      if (sum >= share) break;
    }
    atomicMin(&s_waves, k);
  }
  __syncthreads();
  const int waves = ctas > 0 ? s_waves : 0;
  // what each CTA lacks after them (at least a unit), and its place in the rest of the line
  int64_t lacks = 0;
  if (tid < ctas) {
    lacks = share;
    for (int k = 0; k < waves; ++k) lacks -= big_size((k * ctas + tid) / p.Hkv);
  }
  if (tid < kServeMaxGrid) {  // whole warps
    int64_t x = lacks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    s_from[tid] = x - lacks;
  }
  __syncthreads();
  int64_t rest = 0;  // where the rest begins
  if (tid < kServeMaxGrid) {
    const int first = waves * ctas;
    if (first < n_items) rest = s_big_at[first / p.Hkv] * p.Hkv + (int64_t)(first % p.Hkv) * big_size(first / p.Hkv);
    else rest = line;
    int64_t before = rest;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    s_from[tid] += before;
  }
  __syncthreads();
  // the big tile and kv head at a place of the line
  auto place = [&](int64_t at, int& j, int& g, int64_t& start, int& n) {
    int lo = 0, hi = n_big;  // the last j with s_big_at[j] * Hkv <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_big_at[mid] * p.Hkv <= at) lo = mid;
      else hi = mid;
    }
    j = lo;
    n = big_size(lo);
    g = (int)((at - s_big_at[lo] * p.Hkv) / n);
    start = s_big_at[lo] * p.Hkv + (int64_t)g * n;
  };
  auto write_item = [&](ChunkItem* item, const PlanTile& r, int u0, int u1, int slot, int g) {
    const int n = s_n[r.b], len = s_len[r.b];
    int4* dst = reinterpret_cast<int4*>(item);
    dst[0] = make_int4(r.b, r.row0, u0, u1);
    dst[1] = make_int4(slot, s_q0[r.b], n, len);
    dst[2] = make_int4(first_key_of(p, n, len), g, 0, 0);
  };
  if (tid < ctas) {
    int k = 0;
    for (; k < waves; ++k) {
      const int i = k * ctas + tid;
      const PlanTile r = tile_of(s_big[i / p.Hkv]);
      write_item(p.big + tid * kBigPieces + k, r, r.u0, r.u1, -1, i % p.Hkv);
    }
    const int64_t begin = s_from[tid], end = min(line, begin + lacks);
    int64_t at = begin;
    while (at < end && k < kBigPieces) {
      int j, g, n;
      int64_t start;
      place(at, j, g, start, n);
      const PlanTile r = tile_of(s_big[j]);
      const int64_t stop = min(end, start + n);
      const bool whole = at == start && stop == start + n;
      write_item(p.big + tid * kBigPieces + k, r, r.u0 + (int)(at - start), r.u0 + (int)(stop - start),
                 whole ? -1 : 2 * tid + (at == begin ? 0 : 1), g);
      // the tile's first cut lies at the end of this share: it is joined from here on
      if (!whole && at == start) {
        int lo = tid, hi = ctas;  // the CTA of the tile's last unit: the last with s_from <= it
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_from[mid] <= start + n - 1) lo = mid;
          else hi = mid;
        }
        ChunkSplit sp;
        sp.b = r.b;
        sp.row0 = r.row0;
        sp.g = g;
        sp.c0 = tid;
        sp.c1 = lo;
        sp.first = at == begin ? 0 : 1;
        sp.pad0 = sp.pad1 = 0;
        p.splits[atomicAdd(&s_splits, 1)] = sp;
      }
      at = stop;
      ++k;
    }
    p.big_count[tid] = k;
  }
  for (int t = tid; t < tiles; t += kPlanThreads) {
    const PlanTile r = tile(t);
    const int n = r.u1 - r.u0;
    if (!is_big(n)) write_item(p.items + atomicAdd(&s_bin[bin_of(n)], 1), r, r.u0, r.u1, -1, 0);
  }
  __syncthreads();
  if (tid == 0)
    *reinterpret_cast<int4*>(p.plan) = make_int4(small, s_splits, ctas, ctas < p.grid ? ctas : 0);
}

// CTA 0 makes the plan (but for light calls); the others (if there are new rows) append: CTA 1 + b + B y takes sequence b, a
// thread per 16-byte chunk of a row.
__global__ void __launch_bounds__(kPlanThreads) chunk_prepare(const __grid_constant__ ServeAttnParams p, int elem) {
  pdl_launch_dependents();
  extern __shared__ int s_seq[];  // [B + 1], [B], [B], [B]
  if (blockIdx.x == 0 && p.light) {  // no plan: the status only
    if (threadIdx.x == 0) status_clear_for_launch(p.status);
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) {
      const SeqInfo s = seq_info(p, b);
      if (s.bad) status_report(p.status, s.bad);
    }
    return;
  }
  if (blockIdx.x == 0) {
    plan_body(p, s_seq, s_seq + p.B + 1, s_seq + 2 * p.B + 1, s_seq + 3 * p.B + 1);
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

// Merge of cut tiles: a unit of work is (cut tile of a kv head, block of 128 rows, 8 columns),
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
  const int total = __ldcg(&p.plan->n_splits) * blocks * chunks;
  for (int x = blockIdx.x * groups + sub; x < total; x += gridDim.x * groups) {
    const int d0 = x % chunks * kChunkMergeCols;
    const int m = x / chunks % blocks * rows_per + m_in;
    const int4* sp = reinterpret_cast<const int4*>(p.splits + x / chunks / blocks);
    const int4 w0 = __ldcg(sp);
    const int2 w1 = __ldcg(reinterpret_cast<const int2*>(sp + 1));
    const int b = w0.x, row0 = w0.y, g = w0.z, pieces = w1.x - w0.w + 1;
    const SeqInfo s = seq_info(p, b);
    if (row0 + m >= s.n * p.G) continue;
    // record of piece i: 2 c0 + first, then 2 (c0 + i)
    const float2* ml = p.part_ml + (int64_t)(2 * w0.w) * p.row_tile + m;
    const float* src = p.part_o + ((int64_t)(2 * w0.w) * p.D + d0) * p.row_tile + m;
    auto rec = [&](int i) { return (int64_t)(i == 0 ? w1.y : 2 * i) * p.row_tile; };
    float M = neg_inf();
#pragma unroll 8
    for (int i = 0; i < pieces; ++i) M = fmaxf(M, __ldcg(ml + rec(i)).x);
    float L = 0.f, acc[kChunkMergeCols];
#pragma unroll
    for (int e = 0; e < kChunkMergeCols; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < pieces; i0 += kMergeBatch) {
      float2 a[kMergeBatch];
      float v[kMergeBatch][kChunkMergeCols];
#pragma unroll
      for (int u = 0; u < kMergeBatch; ++u) {
        const bool in = i0 + u < pieces;
        a[u] = in ? __ldcg(ml + rec(i0 + u)) : make_float2(neg_inf(), 0.f);
#pragma unroll
        for (int e = 0; e < kChunkMergeCols; ++e) v[u][e] = in ? __ldcg(src + rec(i0 + u) * p.D + e * p.row_tile) : 0.f;
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
    const int64_t off = o_offset(p, s, g, row0 + m) + d0;
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
// Two records per share of cut tiles.
constexpr size_t kChunkRecords = 2 * (size_t)kServeMaxGrid;

static void chunk_layout(int64_t T, int G, int B, int D, int row_tile, size_t (&at)[8]) {
  at[0] = 256;                                                              // plan
  at[1] = at[0] + 256;                                                      // pieces of cut tiles per CTA
  at[2] = up256(at[1] + kServeMaxGrid * sizeof(int32_t));                   // those pieces
  at[3] = up256(at[2] + (size_t)kServeMaxGrid * kBigPieces * sizeof(ChunkItem));  // small tiles
  at[4] = up256(at[3] + (size_t)chunk_max_tiles(T, G, B, row_tile) * sizeof(ChunkItem));  // cut tiles
  at[5] = up256(at[4] + kServeMaxGrid * sizeof(ChunkSplit));                // (m, l)
  at[6] = up256(at[5] + kChunkRecords * row_tile * sizeof(float2));         // o
  at[7] = up256(at[6] + kChunkRecords * row_tile * (size_t)D * sizeof(float));
}
size_t chunk_workspace_bytes(int64_t T, int G, int B, int D, int row_tile) {
  size_t at[8];
  chunk_layout(T, G, B, D, row_tile, at);
  return at[7];
}
void chunk_workspace_carve(void* ws, ServeAttnParams* p) {
  size_t at[8];
  chunk_layout(p->T, p->G, p->B, p->D, p->row_tile, at);
  char* b = reinterpret_cast<char*>(ws);
  p->status = reinterpret_cast<uint32_t*>(b);
  p->plan = reinterpret_cast<ChunkPlan*>(b + at[0]);
  p->big_count = reinterpret_cast<int32_t*>(b + at[1]);
  p->big = reinterpret_cast<ChunkItem*>(b + at[2]);
  p->items = reinterpret_cast<ChunkItem*>(b + at[3]);
  p->splits = reinterpret_cast<ChunkSplit*>(b + at[4]);
  p->part_ml = reinterpret_cast<float2*>(b + at[5]);
  p->part_o = reinterpret_cast<float*>(b + at[6]);
  p->max_tiles = (int)chunk_max_tiles(p->T, p->G, p->B, p->row_tile);
}

cudaError_t launch_chunk_prepare(const ServeAttnParams& p, int elem_bytes, cudaStream_t stream) {
  const int smem = (4 * p.B + 1) * (int)sizeof(int);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(chunk_prepare), smem);
  if (e != cudaSuccess) return e;
  unsigned grid = 1;
  if (p.k_new) {  // about 2400 CTAs at most, one per sequence at least
    const int64_t want = ((int64_t)p.max_q * p.Hkv * (p.D * elem_bytes / 16) + kPlanThreads - 1) / kPlanThreads;
    const int64_t most = (2400 + p.B - 1) / p.B;
    grid += (unsigned)p.B * (unsigned)(want < most ? want : most);
  }
  chunk_prepare<<<grid, kPlanThreads, smem, stream>>>(p, elem_bytes);
  return cudaGetLastError();
}
cudaError_t launch_chunk_merge(const ServeAttnParams& p, cudaStream_t stream) {
  return launch_dependent(chunk_merge, dim3(4 * p.grid), dim3(kMergeThreads), 0, stream, 0u, p);
}

}  // namespace specv
