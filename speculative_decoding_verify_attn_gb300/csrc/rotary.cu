// Rotary positions of a batch's new tokens.
//
// A pair (a, b) of a head at position p is turned by 2 pi * frac(p * step / 2^64).  The product modulo 2^64
// is two integer instructions and exact, so a position of a million costs no accuracy and no fp64; its top
// 32 bits, as a signed fraction of half a turn, go to sincospi.
//
// Bound: HBM, each value read and written once.  A CTA takes `tile` tokens: it works their rot / 2 sines and
// cosines out once, in shared memory, for all heads of q and k, then streams the heads, 16 bytes a lane
// (a pair of chunks where the layout pairs the halves), or fewer where rot suits no such access.  Measured, 16384
// tokens of 40 heads of 128 in bf16: 57 us (5.85 TB/s), rot 116 in halves (4 bytes a lane) 104 us; 40 tokens 5 us of
// device time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache_internal.h"
#include "common.cuh"

namespace specv {

constexpr int kRotaryThreads = 256;

// V bytes of a head as floats and back
template <int V>
struct Word;
template <> struct Word<16> { using T = uint4; };
template <> struct Word<8> { using T = uint2; };
template <> struct Word<4> { using T = uint32_t; };
template <> struct Word<2> { using T = uint16_t; };
template <bool F32, int V>
struct Chunk {
  using T = typename Word<V>::T;
  static constexpr int E = F32 ? V / 4 : V / 2;
  float v[E];
  __device__ __forceinline__ void set(const T& w) {
    if constexpr (V == 2) {
      v[0] = __uint_as_float((uint32_t)w << 16);
    } else {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        if constexpr (F32) {
          v[i] = __uint_as_float(u[i]);
        } else {
          v[2 * i] = __uint_as_float(u[i] << 16);
          v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ T get() const {
    T w;
    if constexpr (V == 2) {
      w = (uint16_t)pack_bf16(v[0], 0.f);
    } else {
      uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        if constexpr (F32) u[i] = __float_as_uint(v[i]);
        else u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      }
    }
    return w;
  }
};

// Pairs that a chunk (or, in halves, two chunks) makes, and the place of pair i of a token in shared memory: the
// pairs of neighbouring chunks at equal places of theirs lie side by side, two to 16 bytes, so that a warp
// reads them without conflicts.
template <bool F32, bool PAIRS, int V>
struct Turns {
  static constexpr int N = Chunk<F32, V>::E / (PAIRS ? 2 : 1);
  static __device__ __forceinline__ int at(int i, int chunks) {
    if constexpr (N == 1) return i;
    const int u = i / N, e = i % N;
    return ((e >> 1) * chunks + u) * 2 + (e & 1);
  }
};

__device__ __forceinline__ void turn(const float2 cs, float& a, float& b) {
  const float x = a * cs.x - b * cs.y;
  b = b * cs.x + a * cs.y;
  a = x;
}

template <bool F32, bool PAIRS, int V>
__device__ __forceinline__ void rotate_heads(const RotaryParams& p, const float2* table, const int* s_ok, int t0, int n,
                                             const void* src, int64_t st, int64_t sh, void* dst, int64_t dt, int64_t dh,
                                             int heads, bool copy) {
  using C = Chunk<F32, V>;
  using T = typename C::T;
  constexpr int S = F32 ? 4 : 2, E = C::E, N = Turns<F32, PAIRS, V>::N, kBatch = 4;
  const char* in = reinterpret_cast<const char*>(src);
  char* out = reinterpret_cast<char*>(dst);
  const int half = p.rot / 2, turned = half / N;
  const int per = turned + (copy ? (p.D - p.rot) / E : 0);
  // a thread keeps its place in the head and steps over the rows (token, head), kBatch of them in flight: 16 bytes a
  // lane, 57 us for 16384 rows of 40 heads (two in flight 62, eight 62)
  const int width = min(per, kRotaryThreads), step = kRotaryThreads / width, rows = n * heads;
  const int first = (int)threadIdx.x / width < step ? threadIdx.x / width : rows;
  for (int u = threadIdx.x % width; u < per; u += width) {
    const bool rotates = u < turned;
    const int at = rotates ? u * V : (p.rot + (u - turned) * E) * S;
    for (int r0 = first; r0 < rows; r0 += kBatch * step) {
      T a[kBatch], b[kBatch];
      char* y[kBatch];
      int token[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * step, j = r / heads, h = r - j * heads;
        token[i] = r < rows && s_ok[j] ? j : -1;
        if (token[i] < 0) continue;
        const char* x = in + ((int64_t)(t0 + j) * st + (int64_t)h * sh) * S + at;
        y[i] = out + ((int64_t)(t0 + j) * dt + (int64_t)h * dh) * S + at;
        a[i] = *reinterpret_cast<const T*>(x);
        if (!PAIRS && rotates) b[i] = *reinterpret_cast<const T*>(x + half * S);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (token[i] < 0) continue;
        if (rotates) {
          const float2* cs = table + token[i] * half;
          C v, w;
          v.set(a[i]);
          if (!PAIRS) w.set(b[i]);
          auto pair = [&](int e, const float2 z) {
            if constexpr (PAIRS) turn(z, v.v[2 * e], v.v[2 * e + 1]);
            else turn(z, v.v[e], w.v[e]);
          };
          if constexpr (N == 1) {
            pair(0, cs[u]);
          } else {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
              const float2* z = cs + ((e >> 1) * turned + u) * 2;
              pair(e, z[0]);
              pair(e + 1, z[1]);
            }
          }
          a[i] = v.get();
          if (!PAIRS) *reinterpret_cast<T*>(y[i] + half * S) = w.get();
        }
        *reinterpret_cast<T*>(y[i]) = a[i];
      }
    }
  }
}

template <bool F32, bool PAIRS, int V>
__global__ void __launch_bounds__(kRotaryThreads) rotary(const __grid_constant__ RotaryParams p) {
  extern __shared__ __align__(16) float2 s_table[];  // [tile][rot / 2]
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
    s_table[j * half + Turns<F32, PAIRS, V>::at(u, half / Turns<F32, PAIRS, V>::N)] =
        make_float2(c * p.amplitude, (p.negate ? -s : s) * p.amplitude);
  }
  __syncthreads();
  rotate_heads<F32, PAIRS, V>(p, s_table, s_ok, t0, n, p.q, p.q_st, p.q_sh, p.qo, p.qo_st, p.qo_sh, p.Hq, p.copy_q);
  rotate_heads<F32, PAIRS, V>(p, s_table, s_ok, t0, n, p.k, p.k_st, p.k_sh, p.ko, p.ko_st, p.ko_sh, p.Hkv, p.copy_k);
}

template <bool F32, bool PAIRS, int V>
static cudaError_t launch_width(const RotaryParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)((p.T + p.tile - 1) / p.tile);
  const size_t smem = (size_t)p.tile * (p.rot / 2) * sizeof(float2);
  rotary<F32, PAIRS, V><<<grid, kRotaryThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

// The widest access that divides what is turned (a half, or all pairs) and what is copied.
template <bool F32, bool PAIRS>
static cudaError_t launch_layout(const RotaryParams& p, cudaStream_t stream) {
  const int bytes = (PAIRS ? p.rot : p.rot / 2) * (F32 ? 4 : 2) | (p.D - p.rot) * (F32 ? 4 : 2);
  if (bytes % 16 == 0) return launch_width<F32, PAIRS, 16>(p, stream);
  if (bytes % 8 == 0 || (F32 && PAIRS)) return launch_width<F32, PAIRS, 8>(p, stream);
  if constexpr (!(F32 && PAIRS)) {
    if (bytes % 4 == 0 || F32 || PAIRS) return launch_width<F32, PAIRS, 4>(p, stream);
  }
  if constexpr (!F32 && !PAIRS) return launch_width<F32, PAIRS, 2>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
  if (p.f32) return p.pairs ? launch_layout<true, true>(p, stream) : launch_layout<true, false>(p, stream);
  return p.pairs ? launch_layout<false, true>(p, stream) : launch_layout<false, false>(p, stream);
}

}  // namespace specv
