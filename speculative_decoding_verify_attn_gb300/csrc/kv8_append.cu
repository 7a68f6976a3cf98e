// New K/V rows into the pages of an 8-bit cache.
//
// A warp takes one block of tokens of one head, of K or of V: the largest magnitude of the block's new rows
// gives the exponent the block needs; if the block holds earlier tokens of the sequence it keeps at least
// its own, and where that grows the earlier rows are brought to it; then the new rows are scaled
// (exactly: a power of two), rounded and stored.  A block's rows are therefore in one warp's hands, and
// nothing has to be ordered between warps.
// A lane holds 16 values of a row, so that a store is 16 bytes.  Up to 32 rows of 128 values (bf16) stay in
// registers between the two steps, all loads of them in flight at once; larger blocks are read twice.
// Bound: HBM for prompts (2 or 4 bytes read and 1 written per value), latency for a round's few rows.  Measured: 16K
// rows of 8 heads of 128 from bf16 22 us (4.4 TB/s; a unit is a chain of four trips to memory), 40 rows 5 us of device time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "cache_internal.h"
#include "common.cuh"
#include "kv8_common.cuh"

namespace specv {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;

// 16 values of a row as they lie in memory.
template <bool F32>
struct Raw16 {
  static constexpr int W = F32 ? 4 : 2;
  uint4 w[W];
  __device__ __forceinline__ void load(const void* src, int64_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(src) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __ldg(s + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // value 4 j + i of the 16
  __device__ __forceinline__ void four(int j, float (&v)[4]) const {
    if constexpr (F32) {
      v[0] = __uint_as_float(w[j].x); v[1] = __uint_as_float(w[j].y); v[2] = __uint_as_float(w[j].z); v[3] = __uint_as_float(w[j].w);
    } else {
      const uint32_t a = j & 1 ? w[j >> 1].z : w[j >> 1].x, b = j & 1 ? w[j >> 1].w : w[j >> 1].y;
      v[0] = __uint_as_float(a << 16); v[1] = __uint_as_float(a & 0xffff0000u);
      v[2] = __uint_as_float(b << 16); v[3] = __uint_as_float(b & 0xffff0000u);
    }
  }
  // The largest magnitude and `top`, as the bits of |x| (two halves for bf16): in the order of whole numbers,
  // infinities and NaN come behind all finite values, so two instructions a word do for the usual case.
  __device__ __forceinline__ uint32_t magnitude(uint32_t top) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F32) top = max(top, u[e] & 0x7fffffffu);
        else top = __vmaxu2(top, u[e] & 0x7fff7fffu);
      }
    }
    return top;
  }
  // the same without what is not finite
  __device__ __forceinline__ uint32_t finite_magnitude(uint32_t top) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F32) {
          const uint32_t a = u[e] & 0x7fffffffu;
          top = max(top, a < 0x7f800000u ? a : 0u);
        } else {
          const uint32_t a = u[e] & 0x7fffu, b = u[e] & 0x7fff0000u;
          top = __vmaxu2(top, (a < 0x7f80u ? a : 0u) | (b < 0x7f800000u ? b : 0u));
        }
      }
    }
    return top;
  }
  // the warp's largest, as the bits of a float
  static __device__ __forceinline__ uint32_t join(uint32_t top) {
    if constexpr (!F32) top = max(top << 16, top & 0xffff0000u);
    return __reduce_max_sync(0xffffffffu, top);
  }
  __device__ __forceinline__ uint4 encode(float scale) const {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
      four(j, v);
      u[j] = f32x4_to_e4m3x4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// Blocks that get new tokens.
__device__ __forceinline__ int touched_blocks(const Kv8Params& p, const SeqInfo& s) {
  return s.len > 0 ? (s.len - 1) / p.block - (s.len - s.n) / p.block + 1 : 0;
}

// HOLD: with the way that keeps rows in registers (16K prompt rows 23 us, without it 31); without it the kernel is shorter
// and done sooner (rounds with their attention: 8 sequences of 5 tokens at 16K-32K 106.2 us instead of 106.9, 32 at 1K-4K
// 65.7 and 66.7).
template <bool F32, int D, bool HOLD>
__global__ void __launch_bounds__(kAppendThreads) kv8_append(const __grid_constant__ Kv8Params p, int first) {
  pdl_launch_dependents();
  constexpr int LANES = D / 16, ROWS = 32 / LANES;  // lanes of a row, rows of an instruction
  constexpr int HELD = HOLD ? (F32 ? 4 : 8) : 1;    // of a lane's rows that registers hold (64)
  extern __shared__ int s_pre[];  // [B + 1] blocks before each sequence
  __shared__ int s_sum[kAppendWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (first && blockIdx.x == 0 && tid == 0) status_clear_for_launch(p.status);
  auto report = [&](uint32_t bits) {
    if (first) {
      status_report(p.status, bits);
    } else {
      pdl_wait();  // the kernel before clears the status
      atomicOr(p.status, bits);
    }
  };
  // prefix sums over the sequences: T rows make at most T blocks, but sequences that overlap can claim more
  int run = 0;
  for (int b0 = 0; b0 < p.B; b0 += kAppendThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.B) {
      const SeqInfo s = seq_info(p, b);
      n = touched_blocks(p, s);
      if (s.bad && blockIdx.x == 0) report(s.bad);
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int pre = run;
#pragma unroll
    for (int w = 0; w < kAppendWarps; ++w) {
      if (w < warp) pre += s_sum[w];
      run += s_sum[w];
    }
    if (b < p.B) s_pre[b] = pre + x - n;
    run = min(run, 1 << 26);  // at most 2^22 per sequence: no overflow; nothing valid comes near
  }
  if (tid == 0) s_pre[p.B] = run;
  __syncthreads();

  const int64_t units = (int64_t)run * p.Hkv * 2;
  const int c = lane % LANES, rl = lane / LANES;
  for (int64_t unit = (int64_t)blockIdx.x * kAppendWarps + warp; unit < units; unit += (int64_t)gridDim.x * kAppendWarps) {
    const bool is_v = unit & 1;
    const int g = (int)(unit / 2 % p.Hkv), blk = (int)(unit / 2 / p.Hkv);
    int lo = 0, hi = p.B;  // the last sequence that begins at blk or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= blk) lo = mid;
      else hi = mid;
    }
    const SeqInfo s = seq_info(p, lo);
    const int fresh = s.len - s.n;  // the first new token
    const int t0 = (fresh / p.block + blk - s_pre[lo]) * p.block;
    const int begin = max(t0, fresh), end = min(t0 + p.block, s.len);
    if (blk < s_pre[lo] || begin >= end) continue;  // sequences that overlap by more rows than there can be
    int page, slot;
    page_slot(p, lo, t0, page, slot);
    if (page < 0) {
      if (lane == 0) report((uint32_t)SPEC_STATUS_BAD_PAGE);
      continue;
    }
    const void* src = is_v ? p.v_new : p.k_new;
    const int64_t from = (int64_t)(s.q0 + begin - fresh) * p.new_st + (int64_t)g * p.new_sh + c * 16;
    uint8_t* exp = (is_v ? p.v_exp : p.k_exp) + (int64_t)page * p.exp_sp + (int64_t)g * p.exp_sh + block_of(p, slot);
    uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? p.v : p.k) + (int64_t)page * p.kv_sp + (int64_t)g * p.kv_sh + c * 16;
    const int old = begin > t0 ? clamp_exp(*exp) : 0;
    const int rows = end - begin;
    const bool held = HOLD && rows <= HELD * ROWS;
    Raw16<F32> x[HELD];
    if (held) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if (i * ROWS + rl < rows) x[i].load(src, from + (int64_t)(i * ROWS + rl) * p.new_st);
        else x[i].clear();
      }
    }
    auto largest = [&](auto finite) -> uint32_t {
      uint32_t top = 0u;
      if (held) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) top = finite.value ? x[i].finite_magnitude(top) : x[i].magnitude(top);
      } else {
#pragma unroll 4
        for (int r = rl; r < rows; r += ROWS) {
          Raw16<F32> y;
          y.load(src, from + (int64_t)r * p.new_st);
          top = finite.value ? y.finite_magnitude(top) : y.magnitude(top);
        }
      }
      return Raw16<F32>::join(top);
    };
    uint32_t amax = largest(std::false_type{});
    if (__builtin_expect(amax >= 0x7f800000u, 0)) amax = largest(std::true_type{});
    const int e = max(old, needed_exp(__uint_as_float(amax)));
    if (begin > t0 && e > old) {
      const float down = exp2_whole(old - e >= -126 ? old - e : -126);
      for (int r = rl; r < begin - t0; r += ROWS) {
        uint4* at = reinterpret_cast<uint4*>(dst + (int64_t)(slot + r) * p.kv_st);
        uint4 w = *at;
        uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a, b;
          e4m3x4_to_f16x4(u[i], a, b);
          const float2 x = f16x2_to_f32x2(a), y = f16x2_to_f32x2(b);
          u[i] = f32x4_to_e4m3x4(x.x * down, x.y * down, y.x * down, y.y * down);
        }
        *at = w;
      }
    }
    const float scale = exp2_whole(127 - e);
    uint8_t* to = dst + (int64_t)(slot + begin - t0) * p.kv_st;
    if (held) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (i * ROWS + rl < rows) *reinterpret_cast<uint4*>(to + (int64_t)(i * ROWS + rl) * p.kv_st) = x[i].encode(scale);
    } else {
#pragma unroll 4
      for (int r = rl; r < rows; r += ROWS) {
        Raw16<F32> y;
        y.load(src, from + (int64_t)r * p.new_st);
        *reinterpret_cast<uint4*>(to + (int64_t)r * p.kv_st) = y.encode(scale);
      }
    }
    __syncwarp();
    if (lane == 0) *exp = (uint8_t)e;
  }
  // the kernel before (a plan) is none of the append's business but for the status; what follows is ordered behind
  // this grid alone, so it is not over before that kernel
  if (!first) pdl_wait();
}

template <bool F32, int D, bool HOLD>
static cudaError_t launch_append(const Kv8Params& p, bool first, int64_t units, cudaStream_t stream) {
  const int smem = (p.B + 1) * (int)sizeof(int);
  const int64_t want = (units + kAppendWarps - 1) / kAppendWarps;
  // one wave (registers leave four CTAs an SM): more CTAs work the sequences out anew, 27 us against 25 for 16K rows
  const unsigned grid = (unsigned)(want < 4 * p.grid ? want : 4 * p.grid);
  if (first) {
    kv8_append<F32, D, HOLD><<<grid, kAppendThreads, smem, stream>>>(p, 1);
    return cudaGetLastError();
  }
  return launch_dependent(kv8_append<F32, D, HOLD>, dim3(grid), dim3(kAppendThreads), smem, stream, 0u, p, 0);
}

// Few units (block, head, K or V) are a round's: their latency counts, not their bytes.
constexpr int64_t kAppendFewUnits = 1024;
template <bool F32, int D>
static cudaError_t launch_append_d(const Kv8Params& p, bool first, cudaStream_t stream) {
  // at most T / block blocks, and two per sequence with tokens
  const int64_t units = (p.T / p.block + 2 * (int64_t)(p.B < p.T ? p.B : p.T)) * p.Hkv * 2;
  return units <= kAppendFewUnits ? launch_append<F32, D, false>(p, first, units, stream)
                                  : launch_append<F32, D, true>(p, first, units, stream);
}

cudaError_t launch_kv8_append(const Kv8Params& p, bool first, cudaStream_t stream) {
  if (p.src_f32) return p.D == 128 ? launch_append_d<true, 128>(p, first, stream) : launch_append_d<true, 64>(p, first, stream);
  return p.D == 128 ? launch_append_d<false, 128>(p, first, stream) : launch_append_d<false, 64>(p, first, stream);
}

}  // namespace specv
