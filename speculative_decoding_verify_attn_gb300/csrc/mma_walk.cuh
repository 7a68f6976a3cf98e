// Shared by the kernels of small chunks over paged caches (paged_mma.cu, paged8_mma.cu): the walk over units
// of keys, laid end to end over all (sequence, kv head) segments and dealt to the CTAs in equal ranges.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

// Warps of a CTA, and keys of a unit that each of them takes.
template <int WARPS_, int KEYS_>
struct MmaCut {
  static constexpr int WARPS = WARPS_, KEYS = KEYS_, THREADS = WARPS * 32, UNIT = WARPS * KEYS;
};

// Units of a segment of sequence s; its first unit starts at key lo rounded down to a warp's keys.
template <typename CUT>
__device__ __forceinline__ int mma_first(const SeqInfo& s) {
  return s.lo & ~(CUT::KEYS - 1);
}
template <typename CUT>
__device__ __forceinline__ int mma_units(const SeqInfo& s) {
  return s.len > 0 ? (s.len - mma_first<CUT>(s) + CUT::UNIT - 1) / CUT::UNIT : 0;
}

template <int WARPS>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) sm[warp] = v;
  __syncthreads();
  int64_t t = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) t += sm[w];
  return t;
}

__device__ __forceinline__ int64_t mma_per_cta(int64_t total, int grid) {
  const int64_t per = (total + grid - 1) / grid;
  return per < 1 ? 1 : per;
}

// Position in the walk over a CTA's units: unit u of nu of segment (b, g), `left` units to go.
template <typename CUT>
struct MmaWalk {
  int b, g, u, nu;
  int64_t left;
  SeqInfo s;
  __device__ __forceinline__ void step(const ServeAttnParams& p) {
    if (--left <= 0) return;
    if (++u < nu) return;
    u = 0;
    if (++g < p.Hkv) return;
    g = 0;
    do {
      s = seq_info(p, ++b);
      nu = mma_units<CUT>(s);
    } while (nu == 0);
  }
};

// This CTA's units: the walk's start in `ld`, false if there are none.  Whole CTA; the s_ arguments are shared
// memory, `report` takes the flags of bad sequences.  Direct mode: the rows of a bad length become zero.
template <int D, typename CUT, typename Report>
__device__ __forceinline__ bool mma_start(const ServeAttnParams& p, MmaWalk<CUT>& ld, int64_t* s_scan, int& s_b, int64_t& s_cum,
                                          Report report) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  if (p.direct) {
    ld.b = cta / p.Hkv;
    ld.g = cta % p.Hkv;
    ld.u = 0;
    ld.s = seq_info(p, ld.b);
    ld.nu = mma_units<CUT>(ld.s);
    ld.left = ld.nu;
    if (ld.s.bad && ld.g == 0 && tid == 0) report(ld.s.bad);
    if (ld.nu == 0) {  // no keys: zeros for the rows of a bad length
      for (int i = tid; i < ld.s.n * p.G * D; i += CUT::THREADS) {
        const int64_t off = o_offset(p, ld.s, ld.g, i / D) + i % D;
        if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[off] = __float2bfloat16_rn(0.f);
        else reinterpret_cast<float*>(p.o)[off] = 0.f;
      }
      return false;
    }
  } else {
    int64_t mine = 0;
    for (int b = tid; b < p.B; b += CUT::THREADS) {
      const SeqInfo s = seq_info(p, b);
      mine += mma_units<CUT>(s);
      if (s.bad && cta == 0) report(s.bad);
    }
    const int64_t total = block_sum<CUT::WARPS>(mine, s_scan) * p.Hkv;
    const int64_t per = mma_per_cta(total, p.grid);
    const int64_t begin = (int64_t)cta * per;
    if (begin >= total) return false;
    ld.left = min(per, total - begin);
    // the sequence whose units hold `begin`
    int64_t run = 0;
    for (int b0 = 0; b0 < p.B; b0 += CUT::THREADS) {
      const int b = b0 + tid;
      const int64_t n = b < p.B ? (int64_t)mma_units<CUT>(seq_info(p, b)) * p.Hkv : 0;
      int64_t x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = x;
      __syncthreads();
      int64_t pre = run, all = 0;
#pragma unroll
      for (int w = 0; w < CUT::WARPS; ++w) {
        if (w < warp) pre += s_scan[w];
        all += s_scan[w];
      }
      const int64_t excl = pre + x - n;
      if (n > 0 && begin >= excl && begin < excl + n) {
        s_b = b;
        s_cum = excl;
      }
      run += all;
      if (begin < run) break;  // the same for all threads
    }
    __syncthreads();
    ld.b = s_b;
    ld.s = seq_info(p, ld.b);
    ld.nu = mma_units<CUT>(ld.s);
    const int64_t rel = begin - s_cum;
    ld.g = (int)(rel / ld.nu);
    ld.u = (int)(rel % ld.nu);
  }
  return true;
}

}  // namespace specv
