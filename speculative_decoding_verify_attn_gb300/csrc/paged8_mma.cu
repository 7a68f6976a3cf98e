// Attention of small chunks (up to kMmaMaxRows query rows per sequence and kv head) over a paged cache in
// 8 bits: the work of paged_mma.cu, with keys of half the bytes.
//
// Bound: HBM, one read of every visible key's bytes; the units, the warps' private rings, the records and the
// kernel that joins them are paged_mma.cu's.  What differs is how a tile of 16 keys gets to mma.sync:
//   e4m3 is brought to fp16 (exactly) in registers, with one conversion per pair of values, and the products
//   are fp16 x fp16 into fp32.  bf16 would take three instructions a pair and round probabilities to 8 bits
//   instead of 11.
//   K: ldmatrix sees pairs of bytes as 16-bit elements, so a lane gets four neighbouring values of a key's row;
//   the dot product does not mind the order of its terms, so they serve as the columns 2 t, 2 t + 1, 2 t + 8,
//   2 t + 9 of a step of 16, and the query is laid out alike.
//   V: a transposed ldmatrix brings two neighbouring columns of two keys; one byte permutation pairs the keys,
//   and columns 2 r, 2 r + 1 take the places r and r + 8 of the 16 rows of the product.
//   A warp takes 32 keys of a unit at a time, two tiles side by side: twice the independent work per warp, and half
//   the bookkeeping per key.  The query's fragments, the same for all warps, are read from shared memory: in
//   registers they left too few (32 rows of 128: 304 us with them, 115 without).
//   A block's K scale multiplies the tile's scores.  Its V scale 2^ev goes into the exponent of the
//   probabilities, p' = 2^(s + ev - R), with R kept near the largest s + ev: p' then fits fp16 for whatever
//   scales, and weighs keys as they weigh in the output.  The sum of the softmax takes p' 2^-ev, or, where a unit's scales
//   are far from 1, 2^(s - R) (kv8_common.cuh says why).
//   fp16 holds p' <= 2^15 and rounds to steps of 2^-24, so R is set 2^7 below the maximum: what a
//   probability of the largest key's size loses is then below 2^-32 of it.
//   The query's rows are scaled into fp16 by one power of two, undone on the scores together with K's scale (a
//   scale for each row: 20 rows 103 us instead of 98).  Parts below 2^-29 of the largest value lose bits, which
//   moves a score by at most 2^-39 of what the largest query could reach.
// Measured (8 sequences of 16K-32K, 32/8 heads of 128, the join included): 4 rows per kv head 63 us (85% of the copy
// rate), 16 rows 70 us (76%), 20 rows 100 us (70%), 32 rows 109 us; past 16 rows two warps a scheduler leave
// its fixed latencies open.  In rows of 64: 40 us for 4 rows (67%), 71 for 20.  Sums by themselves for scales far from 1
// stand in the loop (16 rows of 128 67 us without them, 4 rows of 64 38.6); in a loop of their own, or a function, they cost as much.
#include <cuda_runtime.h>

#include "cache_internal.h"
#include "common.cuh"
#include "kv8_common.cuh"
#include "launch_cache.h"
#include "mma_walk.cuh"

namespace specv {

// How far a score may lie above the reference, and where the reference is set below the maximum.
constexpr float kRescaleLog2 = 15.0f;
constexpr float kHeadroomLog2 = 7.0f;
// The reference of a row that has seen no key: every score lies above it, and 2^(-inf - it) is 0.
constexpr float kNoReference = -3.402823466e38f;
// A row's largest |q| times scale stays below 2^70; here times log2(e).
constexpr float kMaxQueryLog2 = 1.1805916207174113e21f * kLog2e;

template <int D, int NR>
struct Mma8 {
  // 8 sequences of 16K-32K: 8 and 12 warps 47 and 41 us for 4 rows of 64, 75 and 71 for 20; for rows of 128 the
  // registers of 12 do not suffice beyond 16 rows, and up to there make no difference (71 us)
  static constexpr int kWarps = D == 64 ? kMma8WideWarps : kMma8Warps;
  using Cut = MmaCut<kWarps, kMma8Keys>;
  static constexpr int kStage = kMma8Keys * D * 2;      // a warp's K and V
  static constexpr int kStages = (D == 128 ? 24 : 40) / kWarps;
  // the join buffer: a round's columns of 8 rows of every warp (strides without bank conflicts)
  static constexpr int kCols = D == 64 ? 32 : 64;
  static constexpr int kCmbStride = kCols + 4;
  static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage + (size_t)kWarps * 8 * kCmbStride * 4;
  // Place of chunk c (16 bytes) of row r: eight rows' chunks c lie in eight different groups of banks.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return r * D + ((D == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4);
  }
};

template <int D, int NR>
__global__ void __launch_bounds__(Mma8<D, NR>::Cut::THREADS, 1)
    paged8_mma(const __grid_constant__ Kv8Params p) {
  pdl_launch_dependents();
  if (!p.first) pdl_wait();  // the append
  using M = Mma8<D, NR>;
  using Cut = typename M::Cut;
  constexpr int kWarps = M::kWarps;
  constexpr int KS = D / 16;          // k steps of K Q^T, m tiles of V^T P^T, 16-byte chunks of a row
  constexpr int RPI = 32 / KS;        // rows one cp.async instruction of the warp covers
  constexpr int NS = M::kStages;
  constexpr int STAGE = M::kStage;
  constexpr int KT = kMma8Keys / 16;  // tiles of 16 keys, side by side
  extern __shared__ __align__(256) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ float2 s_ml[kWarps][kMmaMaxRows];
  __shared__ float2 s_scale[kWarps][NS][kMma8Keys];  // of a stage's keys: K's scale, V's exponent
  __shared__ uint2 s_q[NR][KS][32];  // the query's fragments
  __shared__ float s_amax[NR];       // the largest magnitude of 8 rows
  __shared__ int s_pos[NR * 8];      // a row's position
  __shared__ int s_b;
  __shared__ int64_t s_cum;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  float* cmb = reinterpret_cast<float*>(smem + (size_t)kWarps * NS * STAGE);
  if (p.first && cta == 0 && tid == 0) status_clear_for_launch(p.status);
  auto report = [&](uint32_t bits) {
    if (p.first) status_report(p.status, bits);
    else atomicOr(p.status, bits);
  };

  MmaWalk<Cut> ld;
  if (!mma_start<D>(p, ld, s_scan, s_b, s_cum, report)) return;

  // ---- loads: the warp's 32 keys of the unit at `ld`, a lane each for page ids (fetched one unit ahead) and scales
  const uint32_t ring_u32 = smem_u32(smem + (size_t)warp * NS * STAGE);
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(p.k);
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(p.v);
  MmaWalk<Cut> cw = ld;  // the unit in compute
  auto first_key = [&](const MmaWalk<Cut>& w) {
    return mma_first<Cut>(w.s) + w.u * Cut::UNIT + warp * kMma8Keys;
  };
  int page = -1;
  auto look_up = [&]() {
    const int t = first_key(ld) + lane;
    page = -1;
    if (ld.left > 0 && t >= ld.s.lo && t < ld.s.len)
      page = __ldg(p.table + (int64_t)ld.b * p.table_stride + page_of(p, t));
  };
  const int c = lane % KS, rl = lane / KS;
  const uint32_t lane_at = M::at(rl, c);
  const bool whole_pages = (p.page_size & (kMma8Keys - 1)) == 0;
  uint8_t k_byte = 127, v_byte = 127;  // of this lane's key of the unit issued last; they reach s_scale one unit later
  bool seen = false;                   // whether that key lies in [lo, len)
  int scale_stage = -1;
  uint32_t far = 0;  // bit of a stage: V's scales are such that the sum is not taken from the probabilities
  auto issue = [&](int stage) {
    if (scale_stage >= 0) {
      const bool any = __any_sync(0xffffffffu, seen && (v_byte < kFarLow || v_byte > kFarHigh));
      far = (far & ~(1u << scale_stage)) | (uint32_t)any << scale_stage;
      s_scale[warp][scale_stage][lane] = make_float2(exp2_whole(clamp_exp(k_byte) - 127), seen ? (float)(clamp_exp(v_byte) - 127) : neg_inf());
    }
    scale_stage = -1;
    if (ld.left > 0) {
      const int t0 = first_key(ld), t = t0 + lane;
      const uint32_t dst = ring_u32 + stage * STAGE + lane_at;
      const bool in = t >= ld.s.lo && t < ld.s.len;
      const bool good = in && page >= 0 && page < p.num_pages;
      const int slot = t - page_of(p, t) * p.page_size;
      const int64_t row = (int64_t)page * p.kv_sp + (int64_t)slot * p.kv_st + (int64_t)ld.g * p.kv_sh;
      k_byte = v_byte = 127;
      seen = in;
      scale_stage = stage;
      if (good) {
        const int64_t at = (int64_t)page * p.exp_sp + (int64_t)ld.g * p.exp_sh + block_of(p, slot);
        k_byte = p.k_exp[at];
        v_byte = p.v_exp[at];
      } else if (in) {
        report((uint32_t)SPEC_STATUS_BAD_PAGE);
      }
      const bool all = __all_sync(0xffffffffu, good);
      // for rows i * RPI + rl the lane's part of the place is constant and i changes it by an offset and an XOR
      if (whole_pages && all) {  // the usual case: 32 cached tokens of one page
        int64_t off = __shfl_sync(0xffffffffu, row, 0) + (int64_t)rl * p.kv_st + c * 16;
        const int64_t step = p.kv_st * RPI;
#pragma unroll
        for (int i = 0; i < kMma8Keys / RPI; ++i) {
          const uint32_t at = (dst + i * RPI * D) ^ (D == 128 ? ((i * RPI) & 7) << 4 : 0);
          cp_async16(at, kb + off);
          cp_async16(at + kMma8Keys * D, vb + off);
          off += step;
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kMma8Keys / RPI; ++i) {
          const int64_t so = __shfl_sync(0xffffffffu, good ? row : -1, i * RPI + rl);
          const uint32_t at = (dst + i * RPI * D) ^ (D == 128 ? ((i * RPI) & 7) << 4 : 0);
          cp_async16(at, kb + (so < 0 ? 0 : so + c * 16), so >= 0);
          cp_async16(at + kMma8Keys * D, vb + (so < 0 ? 0 : so + c * 16), so >= 0);
        }
      }
      ld.step(p);
      look_up();
    }
    cp_async_commit();
  };
  look_up();
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) issue(i);

  // ---- compute
  const int gid = lane >> 2, tq = lane & 3;
  // places of the fragments' rows: K: matrices (keys 0-7, 8-15) x (chunk, chunk + 1); V alike
  const int frag_row = lane & 15, frag_chunk = lane >> 4;
  float o[NR][KS][4];  // columns d = ks * 16 + 2 gid (e < 2), + 1 (e >= 2) of rows nr * 8 + 2 tq + (e & 1)
  float qs = 0.f;      // what the scores are multiplied by
  float m_run[NR][2], l_run[NR][2];  // the reference R, and the sum of 2^(s - R)
  int stage = 0;
  bool fresh_part = true;
  bool starts_at_begin = true;  // the current part starts where the CTA's range starts
  int part_u0 = cw.u;
  while (true) {
    const int rows = cw.s.n * p.G;
    if (__builtin_expect(fresh_part, 0)) {
      fresh_part = false;
      part_u0 = cw.u;
      // the query's fragments, the same for all warps: warp w makes those of the w-th 8 rows, four neighbouring values
      // of each step of 16, as K's rows come
      const int r = warp * 8 + gid;
      const bool real = warp < NR && r < rows;
      const uint2* src = reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                        (real ? q_offset(p, cw.s, cw.g, r) : 0));
      uint2 raw[KS];
      if (warp < NR) {
        float amax = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          raw[ks] = real ? __ldg(src + ks * 4 + tq) : make_uint2(0u, 0u);
          const uint32_t w[2] = {raw[ks].x, raw[ks].y};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            amax = fmax3(amax, fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u)));
        }
        // a row that is not finite, or beyond what a row may be, must not take the others' bits: it counts as zeros
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (!(amax * p.scale_log2 < kMaxQueryLog2)) {
          amax = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) raw[ks] = make_uint2(0u, 0u);
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
        if (lane == 0) s_amax[warp] = amax;
      }
      __syncthreads();  // the part before has ended with one, too
      float amax = s_amax[0], undo;
#pragma unroll
      for (int nr = 1; nr < NR; ++nr) amax = fmaxf(amax, s_amax[nr]);
      const float up = f16_scale(amax, undo);
      qs = q_factor(undo, p.scale_log2);
      if (warp < NR) {
        if (tq == 0) s_pos[r] = cw.s.len - cw.s.n + r / p.G;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t w[2] = {raw[ks].x, raw[ks].y};
          uint32_t f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            f[i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
          s_q[warp][ks][lane] = make_uint2(f[0], f[1]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nr][ks][e] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m_run[nr][h] = kNoReference;
          l_run[nr][h] = 0.f;
        }
      }
    }
    issue(stage == 0 ? NS - 1 : stage - 1);  // NS - 1 units ahead
    cp_async_wait<NS - 1>();
    __syncwarp();
    const int first_new = cw.s.len - cw.s.n;
    const uint32_t ks_u32 = ring_u32 + stage * STAGE, vs_u32 = ks_u32 + kMma8Keys * D;
    const int key0 = first_key(cw);

    // S^T = K Q^T: 16 keys x 8 rows per tile, the keys on the matrix instruction's 16-row side, so
    // few query rows are padded to 8 instead of 16
    float s[KT][NR][4];  // keys gid (e = 0, 1), gid + 8 (e = 2, 3); rows nr * 8 + 2 tq + (e & 1)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kt][nr][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ks += 2) {
      uint32_t w[KT][4];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        ldmatrix_x4(ks_u32 + kt * 16 * D + M::at(frag_row, ks + frag_chunk), w[kt][0], w[kt][1], w[kt][2], w[kt][3]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 q[NR];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) q[nr] = s_q[nr][ks + i][lane];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          uint32_t a[4];
          e4m3x4_to_f16x4(w[kt][2 * i], a[0], a[2]);
          e4m3x4_to_f16x4(w[kt][2 * i + 1], a[1], a[3]);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) mma_f16_16816(s[kt][nr], a, q[nr].x, q[nr].y);
        }
      }
    }
    // the scores s + ev to the base of 2 (keys outside [lo, len) have ev = -inf).  What is rare below is kept
    // short and out of the way: the loop's instructions do not stay in the nearest cache, and jumps over long
    // pieces of code cost more than the pieces (24 rows: 183 us with them unrolled in place)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const float2 a = s_scale[warp][stage][kt * 16 + gid], b = s_scale[warp][stage][kt * 16 + gid + 8];
      const float ka = qs * a.x, kb = qs * b.x;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[kt][nr][e] = fmaf(s[kt][nr][e], e < 2 ? ka : kb, e < 2 ? a.y : b.y);
    }
    // some row must not see some of these keys: past the first new token, or below the last row's window
    if (__builtin_expect(key0 + 16 * KT > first_new + 1 || (p.window > 0 && key0 < cw.s.len - p.window), 0)) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int last = s_pos[nr * 8 + tq * 2 + h], before = p.window > 0 ? last - p.window : -1;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int t = key0 + kt * 16 + i * 8 + gid;
              if (t > last || t <= before) s[kt][nr][2 * i + h] = neg_inf();
            }
        }
    }
    // the reference moves only when a score lies 2^15 above it, so most units need no exchange between
    // lanes; it is then set 2^7 below the new maximum
    bool over = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(s[0][nr][h], s[0][nr][2 + h]);
        x = fmax3(x, s[1][nr][h], s[1][nr][2 + h]);
        over |= x > m_run[nr][h] + kRescaleLog2;
      }
    if (__builtin_expect(__any_sync(0xffffffffu, over), 0)) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = fmaxf(s[0][nr][h], s[0][nr][2 + h]);
          x = fmax3(x, s[1][nr][h], s[1][nr][2 + h]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m_run[nr][h], x - kHeadroomLog2);
          f[h] = ex2_approx(m_run[nr][h] - mn);
          l_run[nr][h] = scale_sum(l_run[nr][h], m_run[nr][h] - mn, f[h]);
          m_run[nr][h] = mn;
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
    const bool far_stage = far >> stage & 1u;
    if (__builtin_expect(far_stage, 0)) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const float va = fmaxf(s_scale[warp][stage][kt * 16 + gid].y, -64.f);
        const float vb = fmaxf(s_scale[warp][stage][kt * 16 + gid + 8].y, -64.f);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            l_run[nr][i & 1] += ex2_approx(s[kt][nr][i] - m_run[nr][i & 1] - (i < 2 ? va : vb));
      }
    }
    uint32_t pf[KT][NR][2];  // P^T as the B operand: 16 keys x 8 rows
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      // 2^-ev; finite where ev is -inf, whose e is 0
      const float most = far_stage ? 0.f : -kNoReference;
      const float ia = fminf(ex2_approx(-s_scale[warp][stage][kt * 16 + gid].y), most);
      const float ib = fminf(ex2_approx(-s_scale[warp][stage][kt * 16 + gid + 8].y), most);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = ex2_approx(s[kt][nr][i] - m_run[nr][i & 1]);
        l_run[nr][0] = fmaf(e[0], ia, fmaf(e[2], ib, l_run[nr][0]));
        l_run[nr][1] = fmaf(e[1], ia, fmaf(e[3], ib, l_run[nr][1]));
        pf[kt][nr][0] = movmatrix_trans(pack_f16(e[0], e[1]));
        pf[kt][nr][1] = movmatrix_trans(pack_f16(e[2], e[3]));
      }
    }
    // O^T += V^T P^T
#pragma unroll
    for (int ks = 0; ks < KS; ks += 2) {
      uint32_t w[KT][4];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        ldmatrix_x4_trans(vs_u32 + kt * 16 * D + M::at(frag_row, ks + frag_chunk), w[kt][0], w[kt][1], w[kt][2], w[kt][3]);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a[4];
          e4m3x4_to_f16x4(__byte_perm(w[kt][2 * i], 0, 0x3120), a[0], a[1]);
          e4m3x4_to_f16x4(__byte_perm(w[kt][2 * i + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) mma_f16_16816(o[nr][ks + i], a, pf[kt][nr][0], pf[kt][nr][1]);
        }
    }
    __syncwarp();  // every lane has read the stage before it is refilled
    stage = stage == NS - 1 ? 0 : stage + 1;

    // ---- end of the part: join the warps' states
    const bool last = cw.left == 1;
    if (__builtin_expect(cw.u + 1 == cw.nu || last, 0)) {
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
          float top = neg_inf();
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r].x);
          f[h] = ex2_approx(m_run[nr][h] - top);
        }
        // the warps' columns of 8 rows through shared memory; then a warp per row adds them up
        constexpr int E = M::kCols / 32;
        const int r = nr * 8 + (warp & 7), col = lane * E;
        float top = neg_inf(), L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = s_ml[w][r];
          L += scale_sum(v.y, v.x - top, ex2_approx(v.x - top));
        }
        const int up = sum_shift(L);
        const float inv = whole ? (L > 0.f ? 1.f / L : 0.f) : exp2_whole(-up);
        if (!whole && r < rows && warp < 8 && lane == 0)
          p.part_ml[rec * kMmaMaxRows + r] = make_float2(top == kNoReference ? neg_inf() : top + up, L * inv);
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += M::kCols) {
#pragma unroll
          for (int x = 0; x < M::kCols / 16; ++x) {
            float* dst = cmb + (warp * 8 + tq * 2) * M::kCmbStride + x * 16 + gid * 2;
            const float* v = o[nr][c0 / 16 + x];
            *reinterpret_cast<float2*>(dst) = make_float2(v[0] * f[0], v[2] * f[0]);
            *reinterpret_cast<float2*>(dst + M::kCmbStride) = make_float2(v[1] * f[1], v[3] * f[1]);
          }
          __syncthreads();
          if (r < rows && warp < 8) {
            float sum[E];
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float* src = cmb + (w * 8 + warp) * M::kCmbStride + col;
              if constexpr (E == 2) {
                const float2 v = *reinterpret_cast<const float2*>(src);
                sum[0] += v.x;
                sum[1] += v.y;
              } else {
                sum[0] += src[0];
              }
            }
            if (!whole) {
              float* dst = p.part_o + (rec * kMmaMaxRows + r) * D + c0 + col;
              if constexpr (E == 2) *reinterpret_cast<float2*>(dst) = make_float2(sum[0] * inv, sum[1] * inv);
              else dst[0] = sum[0] * inv;
            } else {
              const int64_t off = o_offset(p, cw.s, cw.g, r) + c0 + col;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[off + e] = __float2bfloat16_rn(sum[e] * inv);
                else reinterpret_cast<float*>(p.o)[off + e] = sum[e] * inv;
              }
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

template <int D, int NR>
static cudaError_t launch_mma8(const Kv8Params& p, cudaStream_t stream) {
  using M = Mma8<D, NR>;
  const size_t smem = M::kSmem;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(paged8_mma<D, NR>), (int)smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.direct ? p.B * p.Hkv : p.grid);
  if (p.first) {
    paged8_mma<D, NR><<<grid, M::Cut::THREADS, smem, stream>>>(p);
    e = cudaGetLastError();
  } else {
    e = launch_dependent(paged8_mma<D, NR>, grid, dim3(M::Cut::THREADS), smem, stream, 0u, p);
  }
  return e != cudaSuccess || p.direct ? e : launch_paged8_merge(p, M::kWarps, stream);
}

template <int D>
static cudaError_t launch_mma8_d(const Kv8Params& p, cudaStream_t stream) {
  switch ((p.max_q * p.G + 7) / 8) {  // tiles of 8 query rows
    case 1: return launch_mma8<D, 1>(p, stream);
    case 2: return launch_mma8<D, 2>(p, stream);
    case 3: return launch_mma8<D, 3>(p, stream);
    default: return launch_mma8<D, 4>(p, stream);
  }
}

cudaError_t launch_paged8_mma(const Kv8Params& p, cudaStream_t stream) {
  return p.D == 128 ? launch_mma8_d<128>(p, stream) : launch_mma8_d<64>(p, stream);
}

}  // namespace specv
