// Attention of small chunks (up to kMmaMaxRows query rows per sequence and kv head: decode, chain
// verify) over a paged bf16 cache.
//
// Bound: HBM, one read of every visible key's K and V; a group's query rows share it.  Work is cut
// into units of 128 keys, laid end to end over all (sequence, kv head) segments; CTA c takes units
// [c * per, (c + 1) * per), so ragged lengths balance.  A warp owns 16 keys of every unit and runs
// its own pipeline: a private 3-stage ring filled by its own cp.async (16-byte chunks at
// XOR-swizzled places, zeros for slots outside [lo, len)), mma.sync m16n8k16 for K Q^T and V^T P^T, and
// its own running (m, l, O), so no barrier of any kind stands between a warp and its data; the page
// ids of a unit are looked up one unit ahead.  About 128 KB per SM stay in flight.  The eight warps'
// states are joined through shared memory when a segment's part ends.  A part that is the whole
// segment writes o; others leave a record for the merge kernel (a programmatic dependent).
// Short segments (direct mode) are one CTA each and need no merge launch.
// cp.async rather than TMA: a page may be any number of tokens in any layout, and the copies of an
// SM's tensor-memory-access unit complete at a rate set by their number, which small pages multiply.
//
// Measured, 8 sequences of 16K-32K, 32/8 heads of 128: one token each 115 us (6.2 TB/s), five 155 us
// (6.0 TB/s), eight 157 us (5.2 TB/s, the two warps of a scheduler no longer hide each other's latency);
// 8 segments of 300 keys 7.5 us of device time.
//
// Append: a new token's row is read from k_new / v_new and also stored into its slot by the warp
// that owns the key; no CTA reads that slot in this call, so nothing has to be ordered.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_cache.h"
#include "mma_walk.cuh"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

constexpr int kMmaWarps = 8;
constexpr int kMmaThreads = kMmaWarps * 32;
using MmaCut16 = MmaCut<kMmaWarps, kMmaUnit / kMmaWarps>;
constexpr int kMmaStages = 3;
constexpr int kMmaCmbStride = 68;  // floats per row of the 64-column join buffer (conflict-free)
constexpr int kMmaCmbBytes = kMmaWarps * 8 * kMmaCmbStride * 4;
constexpr float kMmaRescaleLog2 = 8.0f;

__host__ __device__ constexpr int mma_stage_bytes(int D) { return 16 * D * 2 * 2; }  // a warp's K and V
__host__ __device__ constexpr size_t mma_smem_bytes(int D) {
  return (size_t)kMmaWarps * kMmaStages * mma_stage_bytes(D) + kMmaCmbBytes;
}

template <int D, int NR>
__global__ void __launch_bounds__(kMmaThreads, 1) paged_mma(const __grid_constant__ ServeAttnParams p) {
  pdl_launch_dependents();
  constexpr int KS = D / 16;        // k steps of K Q^T, m tiles of V^T P^T
  constexpr int CH = D / 8;         // 16-byte chunks of a row
  constexpr int RPI = 32 / CH;      // rows one cp.async instruction of the warp covers
  constexpr int STAGE = mma_stage_bytes(D);
  extern __shared__ __align__(256) uint8_t smem[];
  __shared__ int64_t s_scan[kMmaWarps];
  __shared__ float2 s_ml[kMmaWarps][kMmaMaxRows];
  __shared__ int s_b;
  __shared__ int64_t s_cum;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  float* cmb = reinterpret_cast<float*>(smem + (size_t)kMmaWarps * kMmaStages * STAGE);
  if (cta == 0 && tid == 0) status_clear_for_launch(p.status);

  // ---- this CTA's units
  MmaWalk<MmaCut16> ld;
  if (!mma_start<D>(p, ld, s_scan, s_b, s_cum, [&](uint32_t bits) { status_report(p.status, bits); })) return;

  // ---- loads: the warp's 16 keys of the unit at `ld`, with their page ids fetched one unit ahead
  uint8_t* ring = smem + (size_t)warp * kMmaStages * STAGE;
  const uint32_t ring_u32 = smem_u32(ring);
  const __nv_bfloat16* kb = reinterpret_cast<const __nv_bfloat16*>(p.k);
  const __nv_bfloat16* vb = reinterpret_cast<const __nv_bfloat16*>(p.v);
  const __nv_bfloat16* knew = reinterpret_cast<const __nv_bfloat16*>(p.k_new);
  const __nv_bfloat16* vnew = reinterpret_cast<const __nv_bfloat16*>(p.v_new);
  MmaWalk<MmaCut16> cw = ld;  // the unit in compute
  int page = -1;
  auto look_up = [&]() {  // page id of this lane's key (lanes 16-31 repeat lanes 0-15)
    const int t = (ld.s.lo & ~15) + ld.u * kMmaUnit + warp * 16 + (lane & 15);
    page = -1;
    if (ld.left > 0 && t >= ld.s.lo && t < ld.s.len)
      page = __ldg(p.table + (int64_t)ld.b * p.table_stride + page_of(p, t));
  };
  // chunk c of row r at chunk c ^ (r & 7): for r = i * RPI + lane / CH the lane's part of the place
  // is constant and i changes address bits by XOR and row offset
  const int c = lane % CH, rl = lane / CH;
  const uint32_t lane_at = rl * (D * 2) + ((c ^ rl) << 4);
  auto issue = [&](int stage) {
    if (ld.left > 0) {
      const int t0 = (ld.s.lo & ~15) + ld.u * kMmaUnit + warp * 16;
      const int first_new = ld.s.len - ld.s.n;
      const uint32_t dst = ring_u32 + stage * STAGE;
      const int64_t head = (int64_t)ld.g * p.kv_sh;
      // the usual case: 16 cached tokens of one page
      if ((p.page_size & 15) == 0 && t0 >= ld.s.lo && t0 + 16 <= (knew ? first_new : ld.s.len) && page >= 0 &&
          page < p.num_pages) {
        const int64_t off = (int64_t)page * p.kv_sp + (int64_t)(t0 - page_of(p, t0) * p.page_size + rl) * p.kv_st + head + c * 8;
        const __nv_bfloat16 *ks = kb + off, *vs = vb + off;
        const int64_t step = p.kv_st * RPI;
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const uint32_t at = dst + ((lane_at + i * RPI * (D * 2)) ^ (((i * RPI) & 7) << 4));
          cp_async16(at, ks);
          cp_async16(at + 16 * D * 2, vs);
          ks += step;
          vs += step;
        }
      } else {
        const int t = t0 + (lane & 15);
        const bool in = t >= ld.s.lo && t < ld.s.len;
        const bool good = in && page >= 0 && page < p.num_pages;
        const int64_t slot = good ? (int64_t)page * p.kv_sp + (int64_t)(t - page_of(p, t) * p.page_size) * p.kv_st + head : 0;
        const bool fresh = knew != nullptr && in && t >= first_new;
        const int64_t src = fresh ? (int64_t)(ld.s.q0 + t - first_new) * p.new_st + (int64_t)ld.g * p.new_sh : slot;
        const int kind = fresh ? 2 : (good ? 1 : 0);
        if (in && !good) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_PAGE);
        __syncwarp();
        const bool any_new = __any_sync(0xffffffffu, fresh);
#pragma unroll 1
        for (int i = 0; i < 16 / RPI; ++i) {
          const int r = i * RPI + rl;
          const int64_t so = __shfl_sync(0xffffffffu, src, r);
          const int sk = __shfl_sync(0xffffffffu, kind, r);
          const uint32_t at = dst + r * (D * 2) + ((c ^ (r & 7)) << 4);
          cp_async16(at, (sk == 2 ? knew : kb) + so + c * 8, sk != 0);
          cp_async16(at + 16 * D * 2, (sk == 2 ? vnew : vb) + so + c * 8, sk != 0);
          if (any_new) {  // store the new rows into their slots
            const int64_t to = __shfl_sync(0xffffffffu, slot, r);
            if (__shfl_sync(0xffffffffu, (int)(fresh && good), r)) {
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.k) + to + c * 8) =
                  __ldg(reinterpret_cast<const uint4*>(knew + so + c * 8));
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.v) + to + c * 8) =
                  __ldg(reinterpret_cast<const uint4*>(vnew + so + c * 8));
            }
          }
        }
      }
      ld.step(p);
      look_up();
    }
    cp_async_commit();
  };
  look_up();
  issue(0);
  issue(1);

  // ---- compute
  const int gid = lane >> 2, tq = lane & 3;
  const float sc = p.scale_log2;
  // places of the fragments' rows in a stage (its K, then its V): chunk x of the row is reached by
  // XOR with x << 4
  const uint32_t k_at = (lane & 15) * (D * 2) + (((lane >> 4) ^ (lane & 7)) << 4);
  const uint32_t v_at = 16 * D * 2 + ((lane & 7) + ((lane >> 4) << 3)) * (D * 2) + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  uint32_t qf[NR][KS][2];
  float o[NR][KS][4];  // columns d = ks * 16 + gid (+ 8) of rows nr * 8 + 2 tq (+ 1)
  float m_run[NR][2], l_run[NR][2];
  int stage = 0;
  bool fresh_part = true;
  bool starts_at_begin = true;  // the current part starts where the CTA's range starts
  int part_u0 = cw.u;
  while (true) {
    const int rows = cw.s.n * p.G;
    if (fresh_part) {
      fresh_part = false;
      part_u0 = cw.u;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const int r = nr * 8 + gid;
        const bool real = r < rows;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                                (real ? q_offset(p, cw.s, cw.g, r) : 0));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[nr][ks][0] = real ? __ldg(src + ks * 8 + tq) : 0u;
          qf[nr][ks][1] = real ? __ldg(src + ks * 8 + 4 + tq) : 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nr][ks][e] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m_run[nr][h] = neg_inf();
          l_run[nr][h] = 0.f;
        }
      }
    }
    issue(stage == 0 ? 2 : stage - 1);  // two units ahead
    cp_async_wait<2>();
    __syncwarp();
    const uint32_t ks_u32 = ring_u32 + stage * STAGE;
    const int key0 = (cw.s.lo & ~15) + cw.u * kMmaUnit + warp * 16;

    // S^T = K Q^T: 16 keys x 8 rows per tile, the keys on the matrix instruction's 16-row side, so
    // few query rows are padded to 8 instead of 16
    float s[NR][4];  // keys gid (e = 0, 1), gid + 8 (e = 2, 3); rows nr * 8 + 2 tq + (e & 1)
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nr][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[4];
      ldmatrix_x4((ks_u32 + k_at) ^ (ks << 5), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) mma_bf16_16816(s[nr], a, qf[nr][ks][0], qf[nr][ks][1]);
    }
    // keys some row must not see: past the first new token, below the last row's window, or slots
    // outside [lo, len)
    const int first_new = cw.s.len - cw.s.n;
    if (key0 + 16 > first_new || key0 < cw.s.lo || (p.window > 0 && key0 < cw.s.len - p.window)) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pos = first_new + (nr * 8 + tq * 2 + (e & 1)) / p.G;
          const int t = key0 + gid + (e & 2) * 4;
          const bool vis = t <= pos && t < cw.s.len && t >= cw.s.lo && (p.window <= 0 || t > pos - p.window);
          if (!vis) s[nr][e] = neg_inf();
        }
    }
    // the reference maximum moves only when a score exceeds it by more than 2^8 (P stays below 2^8,
    // and the final division removes the reference), so most units need no exchange between lanes
    bool over = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = fmaxf(s[nr][h], s[nr][2 + h]);
        over |= x != neg_inf() && x * sc > m_run[nr][h] + kMmaRescaleLog2;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = fmaxf(s[nr][h], s[nr][2 + h]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = x == neg_inf() ? m_run[nr][h] : fmaxf(m_run[nr][h], x * sc);
          f[h] = m_run[nr][h] == neg_inf() ? 0.f : ex2_approx(m_run[nr][h] - mn);
          m_run[nr][h] = mn;
          l_run[nr][h] *= f[h];
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          o[nr][ks][0] *= f[0];
          o[nr][ks][1] *= f[1];
          o[nr][ks][2] *= f[0];
          o[nr][ks][3] *= f[1];
        }
      }
    }
    uint32_t pf[NR][2];  // P^T as the B operand: 16 keys x 8 rows
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m = m_run[nr][i & 1];
        e[i] = ex2_approx(fmaf(s[nr][i], sc, m == neg_inf() ? 0.f : -m));
      }
      l_run[nr][0] += e[0] + e[2];
      l_run[nr][1] += e[1] + e[3];
      pf[nr][0] = movmatrix_trans(pack_bf16(e[0], e[1]));
      pf[nr][1] = movmatrix_trans(pack_bf16(e[2], e[3]));
    }
    // O^T += V^T P^T
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[4];
      ldmatrix_x4_trans((ks_u32 + v_at) ^ (ks << 5), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) mma_bf16_16816(o[nr][ks], a, pf[nr][0], pf[nr][1]);
    }
    __syncwarp();  // every lane has read the stage before it is refilled
    stage = stage == kMmaStages - 1 ? 0 : stage + 1;

    // ---- end of the part: join the warps' states
    const bool last = cw.left == 1;
    if (cw.u + 1 == cw.nu || last) {
      const bool whole = part_u0 == 0 && cw.u + 1 == cw.nu;
      const int64_t rec = 2 * (int64_t)cta + (starts_at_begin ? 0 : 1);
      starts_at_begin = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float l = l_run[nr][h];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          if (gid == 0) s_ml[warp][nr * 8 + tq * 2 + h] = make_float2(m_run[nr][h], l);
        }
      __syncthreads();
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        if (nr * 8 >= rows) break;
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = nr * 8 + tq * 2 + h;
          float M = neg_inf();
#pragma unroll
          for (int w = 0; w < kMmaWarps; ++w) M = fmaxf(M, s_ml[w][r].x);
          f[h] = m_run[nr][h] == neg_inf() ? 0.f : ex2_approx(m_run[nr][h] - M);
        }
        // the warps' columns of 8 rows x 64 columns through shared memory; then a warp per row adds
        // them up, two columns per lane
        const int r = nr * 8 + warp, col = lane * 2;
        float M = neg_inf(), L = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) M = fmaxf(M, s_ml[w][r].x);
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) {
          const float2 v = s_ml[w][r];
          L += v.x == neg_inf() ? 0.f : ex2_approx(v.x - M) * v.y;
        }
        const float inv = whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f;
        if (!whole && r < rows && lane == 0) p.part_ml[rec * kMmaMaxRows + r] = make_float2(M, L);
#pragma unroll
        for (int c4 = 0; c4 < D / 64; ++c4) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float* dst = cmb + (warp * 8 + tq * 2) * kMmaCmbStride + x * 16 + gid;
            const float* v = o[nr][c4 * 4 + x];
            dst[0] = v[0] * f[0];
            dst[kMmaCmbStride] = v[1] * f[1];
            dst[8] = v[2] * f[0];
            dst[kMmaCmbStride + 8] = v[3] * f[1];
          }
          __syncthreads();
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kMmaWarps; ++w) {
            const float2 v = *reinterpret_cast<const float2*>(cmb + (w * 8 + warp) * kMmaCmbStride + col);
            sum.x += v.x;
            sum.y += v.y;
          }
          if (r < rows) {
            if (whole) {
              const int64_t off = o_offset(p, cw.s, cw.g, r) + c4 * 64 + col;
              if (p.o_bf16) {
                __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + off;
                const uint32_t v = pack_bf16(sum.x * inv, sum.y * inv);
                if ((reinterpret_cast<uintptr_t>(dst) & 3u) == 0) {
                  *reinterpret_cast<uint32_t*>(dst) = v;
                } else {
                  reinterpret_cast<uint16_t*>(dst)[0] = (uint16_t)v;
                  reinterpret_cast<uint16_t*>(dst)[1] = (uint16_t)(v >> 16);
                }
              } else {
                float* dst = reinterpret_cast<float*>(p.o) + off;
                dst[0] = sum.x * inv;
                dst[1] = sum.y * inv;
              }
            } else {
              *reinterpret_cast<float2*>(p.part_o + (rec * kMmaMaxRows + r) * D + c4 * 64 + col) = sum;
            }
          }
          __syncthreads();
        }
      }
      fresh_part = true;
    }
    if (last) break;
    cw.step(p);
  }
  cp_async_wait<0>();
}

// Joins the records of the segments that were split over CTAs; zeros for rows of a bad length.
// grid (segments, rows / 8), a warp per row; a batch of records' statistics and values are all in flight
// at once.
constexpr int kMmaMergeBatch = 4;
template <int D, typename CUT>
__global__ void __launch_bounds__(kMmaThreads) paged_mma_merge(const __grid_constant__ ServeAttnParams p) {
  __shared__ int64_t s_scan[kMmaWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv, r = blockIdx.y * kMmaWarps + warp;
  int64_t before = 0, all = 0;
  for (int i = tid; i < p.B; i += kMmaThreads) {
    const int u = mma_units<CUT>(seq_info(p, i));
    all += u;
    if (i < b) before += u;
  }
  const int64_t total = block_sum<kMmaWarps>(all, s_scan) * p.Hkv;
  before = block_sum<kMmaWarps>(before, s_scan) * p.Hkv;
  const SeqInfo s = seq_info(p, b);
  const int nu = mma_units<CUT>(s);
  const int64_t per = mma_per_cta(total, p.grid);
  const int64_t start = before + (int64_t)g * nu;
  const int64_t c0 = start / per;
  const int n = nu > 0 ? (int)((start + nu - 1) / per - c0) + 1 : 0;
  // every CTA waits, those with nothing to join too: what follows in the stream is ordered behind this grid
  // alone, and a grid that has not waited can be over before the attention kernel is
  pdl_wait();
  if (r >= s.n * p.G || n == 1) return;  // n == 1: written by its CTA
  // record i: CTA c0 + i's first, but for c0's second where the segment does not start where c0 does
  const int64_t first = 2 * c0 + (nu > 0 && start % per == 0 ? 0 : 1);
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float M = neg_inf(), L = 0.f;
  for (int i0 = 0; i0 < n; i0 += kMmaMergeBatch) {
    float2 ml[kMmaMergeBatch];
    float v[kMmaMergeBatch][E];
#pragma unroll
    for (int u = 0; u < kMmaMergeBatch; ++u) {
      const int i = i0 + u;
      const int64_t at = (i == 0 ? first : 2 * (c0 + i)) * kMmaMaxRows + r;
      ml[u] = i < n ? __ldcg(&p.part_ml[at]) : make_float2(neg_inf(), 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[u][e] = i < n ? __ldcg(p.part_o + at * D + lane * E + e) : 0.f;
    }
    float m = M;
#pragma unroll
    for (int u = 0; u < kMmaMergeBatch; ++u) m = fmaxf(m, ml[u].x);
    if (m == neg_inf()) continue;
    const float a = M == neg_inf() ? 0.f : exp2f(M - m);
    M = m;
    L *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a;
#pragma unroll
    for (int u = 0; u < kMmaMergeBatch; ++u) {
      const float w = ml[u].x == neg_inf() ? 0.f : exp2f(ml[u].x - m);
      L += w * ml[u].y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const int64_t off = o_offset(p, s, g, r) + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[off + e] = __float2bfloat16_rn(acc[e] * inv);
    else reinterpret_cast<float*>(p.o)[off + e] = acc[e] * inv;
  }
}

size_t mma_workspace_bytes(int D) {
  const size_t recs = 2 * (size_t)kServeMaxGrid * kMmaMaxRows;
  return 256 + recs * (sizeof(float2) + (size_t)D * sizeof(float));
}
void mma_workspace_carve(void* ws, ServeAttnParams* p) {
  char* b = reinterpret_cast<char*>(ws);
  p->status = reinterpret_cast<uint32_t*>(b);
  p->part_ml = reinterpret_cast<float2*>(b + 256);
  p->part_o = reinterpret_cast<float*>(b + 256 + 2 * (size_t)kServeMaxGrid * kMmaMaxRows * sizeof(float2));
}

template <typename CUT>
static cudaError_t launch_merge(const ServeAttnParams& p, cudaStream_t stream) {
  const dim3 grid(p.B * p.Hkv, (unsigned)(p.max_q * p.G + kMmaWarps - 1) / kMmaWarps);
  if (p.D == 128) return launch_dependent(paged_mma_merge<128, CUT>, grid, dim3(kMmaThreads), 0, stream, 0u, p);
  return launch_dependent(paged_mma_merge<64, CUT>, grid, dim3(kMmaThreads), 0, stream, 0u, p);
}
cudaError_t launch_paged8_merge(const ServeAttnParams& p, int warps, cudaStream_t stream) {
  if (warps == kMma8Warps) return launch_merge<MmaCut<kMma8Warps, kMma8Keys>>(p, stream);
  return launch_merge<MmaCut<kMma8WideWarps, kMma8Keys>>(p, stream);
}

template <int D, int NR>
static cudaError_t launch_mma(const ServeAttnParams& p, cudaStream_t stream) {
  const size_t smem = mma_smem_bytes(D);
  auto kern = paged_mma<D, NR>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<p.direct ? p.B * p.Hkv : p.grid, kMmaThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.direct) return e;
  return launch_merge<MmaCut16>(p, stream);
}

template <int D>
static cudaError_t launch_mma_d(const ServeAttnParams& p, cudaStream_t stream) {
  switch ((p.max_q * p.G + 7) / 8) {  // tiles of 8 query rows
    case 1: return launch_mma<D, 1>(p, stream);
    case 2: return launch_mma<D, 2>(p, stream);
    case 3: return launch_mma<D, 3>(p, stream);
    default: return launch_mma<D, 4>(p, stream);
  }
}

cudaError_t launch_paged_mma(const ServeAttnParams& p, cudaStream_t stream) {
  return p.D == 128 ? launch_mma_d<128>(p, stream) : launch_mma_d<64>(p, stream);
}

}  // namespace specv
