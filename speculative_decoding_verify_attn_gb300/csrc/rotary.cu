// Rotary positions of a batch's new tokens.
//
// A pair (a, b) of a head at position p is turned by 2 pi * frac(p * step / 2^64).  The product modulo 2^64
// is two integer instructions and exact, so a position of a million costs no accuracy and no fp64; its top
// 32 bits, as a signed fraction of half a turn, go to sincospi.
//
// Bound: HBM, each value read and written once.  A CTA takes `tile` tokens: it works their rot / 2 sines and
// cosines out once, in shared memory, for all heads of q and k, then streams the heads, 16 bytes a lane
// (a pair of chunks where the layout pairs the halves).  Sizes that no 16-byte access suits go value by
// value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "cache_internal.h"
#include "common.cuh"

namespace specv {

constexpr int kRotaryThreads = 256;

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 16 bytes as floats and back
template <bool F32>
struct Chunk {
  static constexpr int E = F32 ? 4 : 8;
  float v[E];
  __device__ __forceinline__ void load(const void* p) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    if constexpr (F32) {
      v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    uint4 w;
    if constexpr (F32)
      w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      w = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    *reinterpret_cast<uint4*>(p) = w;
  }
};

// One token's sines and cosines: [rot / 2].
__device__ __forceinline__ void turn(const float2 cs, float a, float b, float& x, float& y) {
  x = a * cs.x - b * cs.y;
  y = b * cs.x + a * cs.y;
}

template <bool F32, bool PAIRS, bool VEC>
__device__ __forceinline__ void rotate_heads(const RotaryParams& p, const float2* table, const int* s_ok, int t0, int n,
                                             const void* src, int64_t st, int64_t sh, void* dst, int64_t dt, int64_t dh,
                                             int heads, bool copy) {
  constexpr int S = F32 ? 4 : 2;
  const char* in = reinterpret_cast<const char*>(src);
  char* out = reinterpret_cast<char*>(dst);
  const int half = p.rot / 2;
  if constexpr (VEC) {
    using C = Chunk<F32>;
    constexpr int E = C::E;
    const int turned = PAIRS ? p.rot / E : half / E;
    const int per = turned + (copy ? (p.D - p.rot) / E : 0);
    const int total = n * heads * per;
#pragma unroll 2
    for (int i = threadIdx.x; i < total; i += kRotaryThreads) {
      const int u = i % per, th = i / per, h = th % heads, j = th / heads;
      if (!s_ok[j]) continue;
      const char* x = in + ((int64_t)(t0 + j) * st + (int64_t)h * sh) * S;
      char* y = out + ((int64_t)(t0 + j) * dt + (int64_t)h * dh) * S;
      const float2* cs = table + j * half;
      if (u >= turned) {
        const int at = (p.rot + (u - turned) * E) * S;
        *reinterpret_cast<uint4*>(y + at) = *reinterpret_cast<const uint4*>(x + at);
      } else if (PAIRS) {
        C c;
        c.load(x + u * 16);
#pragma unroll
        for (int e = 0; e < E; e += 2) turn(cs[u * (E / 2) + e / 2], c.v[e], c.v[e + 1], c.v[e], c.v[e + 1]);
        c.store(y + u * 16);
      } else {
        C a, b;
        a.load(x + u * 16);
        b.load(x + half * S + u * 16);
#pragma unroll
        for (int e = 0; e < E; ++e) turn(cs[u * E + e], a.v[e], b.v[e], a.v[e], b.v[e]);
        a.store(y + u * 16);
        b.store(y + half * S + u * 16);
      }
    }
  } else {
    using V = typename std::conditional<F32, float, __nv_bfloat16>::type;
    const int per = half + (copy ? p.D - p.rot : 0);
    const int total = n * heads * per;
    for (int i = threadIdx.x; i < total; i += kRotaryThreads) {
      const int u = i % per, th = i / per, h = th % heads, j = th / heads;
      if (!s_ok[j]) continue;
      const V* x = reinterpret_cast<const V*>(in) + (int64_t)(t0 + j) * st + (int64_t)h * sh;
      V* y = reinterpret_cast<V*>(out) + (int64_t)(t0 + j) * dt + (int64_t)h * dh;
      if (u >= half) {
        y[p.rot + u - half] = x[p.rot + u - half];
        continue;
      }
      const int ia = PAIRS ? 2 * u : u, ib = PAIRS ? 2 * u + 1 : u + half;
      float a, b;
      turn(table[j * half + u], (float)x[ia], (float)x[ib], a, b);
      y[ia] = (V)a;
      y[ib] = (V)b;
    }
  }
}

template <bool F32, bool PAIRS, bool VEC>
__global__ void __launch_bounds__(kRotaryThreads) rotary(const __grid_constant__ RotaryParams p) {
  extern __shared__ float2 s_table[];  // [tile][rot / 2]
  __shared__ int s_seq[kRotaryMaxTile], s_pos[kRotaryMaxTile], s_ok[kRotaryMaxTile];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * p.tile, n = min(p.tile, p.T - t0);
  if (blockIdx.x == 0 && tid == 0) status_clear_for_launch(p.status);
  if (p.positions) {
    if (tid < n) {
      s_pos[tid] = __ldg(p.positions + t0 + tid);
      s_ok[tid] = 1;
    }
  } else {
    // the first sequence that a row belongs to
    if (tid < kRotaryMaxTile) s_seq[tid] = p.B;
    __syncthreads();
    for (int b = tid; b < p.B; b += kRotaryThreads) {
      const int a = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
      if (a < 0 || e < a || e > p.T) {
        if (blockIdx.x == 0) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_RANGE);
        continue;
      }
      for (int j = max(0, a - t0); j < min(n, e - t0); ++j) atomicMin(&s_seq[j], b);
    }
    __syncthreads();
    if (tid < n) {
      const int b = s_seq[tid];
      bool ok = b < p.B;
      if (ok) {
        const int a = __ldg(p.q_start + b), rows = __ldg(p.q_start + b + 1) - a, len = __ldg(p.kv_len + b);
        ok = len >= rows;
        if (!ok) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_KV_LEN);
        s_pos[tid] = len - rows + (t0 + tid - a);
      }
      s_ok[tid] = ok;
    }
  }
  __syncthreads();
  const int half = p.rot / 2;
  for (int i = tid; i < n * half; i += kRotaryThreads) {
    const int j = i / half, u = i - j * half;
    if (!s_ok[j]) continue;
    const unsigned long long phase = (unsigned long long)(long long)s_pos[j] * __ldg(p.steps + u);
    float s, c;
    sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    s_table[i] = make_float2(c * p.amplitude, (p.negate ? -s : s) * p.amplitude);
  }
  __syncthreads();
  rotate_heads<F32, PAIRS, VEC>(p, s_table, s_ok, t0, n, p.q, p.q_st, p.q_sh, p.qo, p.qo_st, p.qo_sh, p.Hq, p.copy_q);
  rotate_heads<F32, PAIRS, VEC>(p, s_table, s_ok, t0, n, p.k, p.k_st, p.k_sh, p.ko, p.ko_st, p.ko_sh, p.Hkv, p.copy_k);
}

template <bool F32, bool PAIRS>
static cudaError_t launch_layout(const RotaryParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)((p.T + p.tile - 1) / p.tile);
  const size_t smem = (size_t)p.tile * (p.rot / 2) * sizeof(float2);
  if (p.vec) rotary<F32, PAIRS, true><<<grid, kRotaryThreads, smem, stream>>>(p);
  else rotary<F32, PAIRS, false><<<grid, kRotaryThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
  if (p.f32) return p.pairs ? launch_layout<true, true>(p, stream) : launch_layout<true, false>(p, stream);
  return p.pairs ? launch_layout<false, true>(p, stream) : launch_layout<false, false>(p, stream);
}

}  // namespace specv
