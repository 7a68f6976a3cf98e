// Chunk attention on the CUDA cores: the fp32 form of the paged and packed operators.
//
// A CTA takes the pieces of the plan in turn: 64 query rows against 64-key tiles, which come by cp.async
// one tile ahead.  Thread (ty, tx) of 16 x 16 holds the scores of rows 4 ty .. 4 ty + 3 and keys
// tx + 16 j, and the output columns 4 tx + 64 j of those rows: per four columns of D a warp reads 12 lines
// of shared memory for 64 FMAs a thread (with two rows a thread, 10 for 32).  Warps whose rows are
// padding do not compute; pieces of up to 8 rows share the keys out over the warps instead.
// fp32 throughout: scores by fp32 FMA, 2^x of the fused difference s * scale - m (the rounding of m is the
// same for the whole row and cancels in the normalisation), running maximum, sum and output in fp32.
// Bound: shared memory and the FMA pipes for long chunks (the tensor cores have no fp32 type; 8 prompts of
// 600 tokens, 32/8 heads of 128, 0.86 ms, 28 TFLOP/s), HBM for few rows (8 sequences of 8K, one token,
// 160 us, 3.3 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_cache.h"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

constexpr int kF32Threads = 256;
constexpr int kF32R = kF32Rows / 16;  // rows per thread
constexpr int kF32Few = 8;            // pieces of at most this many rows split the keys over the warps

template <int D>
constexpr size_t f32_smem_bytes() {
  return sizeof(float) * (kF32Rows * (D + 4) + 2 * kF32Keys * (D + 4) + 2 * kF32Keys * D + kF32Rows * (kF32Keys + 4));
}

template <int D, bool LIGHT>
__global__ void __launch_bounds__(kF32Threads, 1) chunk_attn_f32(const __grid_constant__ ServeAttnParams p) {
  pdl_launch_dependents();
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                                // [64][D + 4]
  float* ks2 = qs + kF32Rows * (D + 4);          // [2][64][D + 4]
  float* vs2 = ks2 + 2 * kF32Keys * (D + 4);     // [2][64][D]
  float* ps = vs2 + 2 * kF32Keys * D;            // [64][64 + 4]
  __shared__ float2 s_ml[8][kF32Few];
  __shared__ int64_t s_off[2][kF32Keys];         // where the keys of a unit lie, -1: zeros
  constexpr int C4 = D / 4, OC = D / 64;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float* q = reinterpret_cast<const float*>(p.q);
  const float* k = reinterpret_cast<const float*>(p.k);
  const float* v = reinterpret_cast<const float*>(p.v);
  __shared__ LightSeqs s_light;
  pdl_wait();  // the plan, and appended rows
  if (LIGHT) light_init(p, s_light);
  PieceList<LIGHT> list;
  list.init(p, &s_light);
  for (int round = 0; round < list.rounds; ++round) {
    const PieceItem it = piece_item(list.fetch(p, round));
    if (it.u0 >= it.u1) continue;
    const int b = it.b, g = it.g, row0 = it.row0, u0 = it.u0, u1 = it.u1, slot = it.slot;
    const SeqInfo s = it.s;
    const int rows = min(kF32Rows, s.n * p.G - row0);
    const int warp_row = (tid >> 5) * 2 * kF32R;  // the warp's first row
    __syncthreads();
    for (int i = tid; i < kF32Rows * C4; i += kF32Threads) {
      const int r = i / C4, c = i % C4;
      const float4 x = r < rows ? *reinterpret_cast<const float4*>(q + q_offset(p, s, g, row0 + r) + c * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(qs + r * (D + 4) + c * 4) = x;
    }
    // unit u + 1 is on its way while unit u is computed; its keys were looked up a unit earlier still
    auto look_up = [&](int u) {
      if (u < u1 && tid < kF32Keys) {
        const int key = u * kF32Keys + tid;
        int64_t off = -1;
        if (key >= s.lo && key < s.len) {
          off = key_offset(p, s, b, g, key);
          if (off < 0) chunk_report<LIGHT>(p, (uint32_t)SPEC_STATUS_BAD_PAGE);
        }
        s_off[u & 1][tid] = off;
      }
    };
    auto issue = [&](int u) {
      if (u < u1) {
        float *kd = ks2 + (u & 1) * kF32Keys * (D + 4), *vd = vs2 + (u & 1) * kF32Keys * D;
        for (int i = tid; i < kF32Keys * C4; i += kF32Threads) {
          const int r = i / C4, c = i % C4;
          const int64_t off = s_off[u & 1][r];
          cp_async16(smem_u32(kd + r * (D + 4) + c * 4), k + (off < 0 ? 0 : off) + c * 4, off >= 0);
          cp_async16(smem_u32(vd + r * D + c * 4), v + (off < 0 ? 0 : off) + c * 4, off >= 0);
        }
      }
      cp_async_commit();
    };
    // four output columns of a row: to o, or as they are into the piece's record
    auto store = [&](int row, int d, float4 x, float inv) {
      const float out[4] = {x.x, x.y, x.z, x.w};
      if (slot >= 0) {
        float* dst = p.part_o + ((int64_t)slot * D + d) * kF32Rows + row;
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e * kF32Rows] = out[e];
      } else {
        const int64_t at = o_offset(p, s, g, row0 + row) + d;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[at + e] = __float2bfloat16_rn(out[e] * inv);
          else reinterpret_cast<float*>(p.o)[at + e] = out[e] * inv;
        }
      }
    };
    look_up(u0);
    __syncthreads();
    issue(u0);
    look_up(u0 + 1);
    if (rows <= kF32Few) {
      // ---- few rows (decode): the warps share the keys of a tile instead of the rows.  Warp w takes keys
      // 8 w ..: lane (row, j) the scores of row lane / 4 and keys 2 j, 2 j + 1, then the warp's
      // lanes 4 output columns each for all rows; the eight states are joined at the end.
      const int warp = tid >> 5, lane = tid & 31, row = lane >> 2, kl = warp * 8 + (lane & 3) * 2;
      float* pw = ps + warp * kF32Few * 8;  // [row][8 keys]
      float m = neg_inf(), l = 0.f;
      float4 acc[kF32Few];
#pragma unroll
      for (int r = 0; r < kF32Few; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int pos = s.len - s.n + (row0 + row) / p.G;
      for (int u = u0; u < u1; ++u) {
        const int key0 = u * kF32Keys;
        const float *ks = ks2 + (u & 1) * kF32Keys * (D + 4), *vs = vs2 + (u & 1) * kF32Keys * D;
        __syncthreads();  // unit u + 1 looked up; the buffers of unit u - 1 are free
        issue(u + 1);
        cp_async_wait<1>();
        __syncthreads();  // unit u has landed, its offsets are free
        look_up(u + 2);
        float x[2] = {0.f, 0.f};
#pragma unroll 8
        for (int c = 0; c < C4; ++c) {
          const float4 qq = *reinterpret_cast<const float4*>(qs + row * (D + 4) + c * 4);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 kk = *reinterpret_cast<const float4*>(ks + (kl + j) * (D + 4) + c * 4);
            x[j] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, x[j]))));
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = key0 + kl + j;
          if (!(t <= pos && t < s.len && (p.window <= 0 || t > pos - p.window))) x[j] = neg_inf();
        }
        float mx = fmaxf(x[0], x[1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m, mx == neg_inf() ? mx : mx * p.scale_log2);
        const float ref = mn == neg_inf() ? 0.f : mn;
        if (__any_sync(0xffffffffu, mn > m)) {
          const float a = m == neg_inf() ? 0.f : exp2f(m - mn);
          l *= a;
#pragma unroll
          for (int r = 0; r < kF32Few; ++r) {
            const float ar = __shfl_sync(0xffffffffu, a, r * 4);
            acc[r].x *= ar;
            acc[r].y *= ar;
            acc[r].z *= ar;
            acc[r].w *= ar;
          }
          m = mn;
        }
        float e[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) e[j] = x[j] == neg_inf() ? 0.f : exp2f(fmaf(x[j], p.scale_log2, -ref));
        l += e[0] + e[1];
        *reinterpret_cast<float2*>(pw + row * 8 + (lane & 3) * 2) = make_float2(e[0], e[1]);
        __syncwarp();
        if (lane * 4 < D) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4*>(vs + (warp * 8 + h * 4 + i) * D + lane * 4);
#pragma unroll
            for (int r = 0; r < kF32Few; ++r) {
              const float4 pp = *reinterpret_cast<const float4*>(pw + r * 8 + h * 4);
              acc[r].x = fmaf(pp.w, v[3].x, fmaf(pp.z, v[2].x, fmaf(pp.y, v[1].x, fmaf(pp.x, v[0].x, acc[r].x))));
              acc[r].y = fmaf(pp.w, v[3].y, fmaf(pp.z, v[2].y, fmaf(pp.y, v[1].y, fmaf(pp.x, v[0].y, acc[r].y))));
              acc[r].z = fmaf(pp.w, v[3].z, fmaf(pp.z, v[2].z, fmaf(pp.y, v[1].z, fmaf(pp.x, v[0].z, acc[r].z))));
              acc[r].w = fmaf(pp.w, v[3].w, fmaf(pp.z, v[2].w, fmaf(pp.y, v[1].w, fmaf(pp.x, v[0].w, acc[r].w))));
            }
          }
        }
        __syncwarp();
      }
      cp_async_wait<0>();
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      __syncthreads();  // every warp is done with the tiles; their memory takes the warps' outputs
      float* os = ks2;  // [warp][row][D]
      if ((lane & 3) == 0) s_ml[warp][row] = make_float2(m, l);
      if (lane * 4 < D)
#pragma unroll
        for (int r = 0; r < kF32Few; ++r) *reinterpret_cast<float4*>(os + (warp * kF32Few + r) * D + lane * 4) = acc[r];
      __syncthreads();
      if (warp < rows) {  // warp w joins row w
        float M = neg_inf(), L = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) M = fmaxf(M, s_ml[w][warp].x);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 ml = s_ml[w][warp];
          const float f = ml.x == neg_inf() ? 0.f : exp2f(ml.x - M);
          L += f * ml.y;
          if (lane * 4 < D) {
            const float4 v = *reinterpret_cast<const float4*>(os + (w * kF32Few + warp) * D + lane * 4);
            x.x = fmaf(f, v.x, x.x);
            x.y = fmaf(f, v.y, x.y);
            x.z = fmaf(f, v.z, x.z);
            x.w = fmaf(f, v.w, x.w);
          }
        }
        if (slot >= 0 && lane == 0) p.part_ml[(int64_t)slot * kF32Rows + warp] = make_float2(M, L);
        if (lane * 4 < D) store(warp, lane * 4, x, L > 0.f ? 1.f / L : 0.f);
      }
      continue;
    }
    float m[kF32R], l[kF32R];
    float4 o[kF32R][OC];
#pragma unroll
    for (int r = 0; r < kF32R; ++r) {
      m[r] = neg_inf();
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < OC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int u = u0; u < u1; ++u) {
      const int key0 = u * kF32Keys;
      const float *ks = ks2 + (u & 1) * kF32Keys * (D + 4), *vs = vs2 + (u & 1) * kF32Keys * D;
      __syncthreads();  // unit u + 1 looked up; the buffers of unit u - 1 are free
      issue(u + 1);
      cp_async_wait<1>();
      __syncthreads();  // unit u has landed, its offsets are free
      look_up(u + 2);
      if (warp_row >= rows) continue;  // rows of padding only
      float x[kF32R][4];
#pragma unroll
      for (int r = 0; r < kF32R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[r][j] = 0.f;
#pragma unroll 2
      for (int c = 0; c < C4; ++c) {
        float4 qq[kF32R];
#pragma unroll
        for (int r = 0; r < kF32R; ++r) qq[r] = *reinterpret_cast<const float4*>(qs + (kF32R * ty + r) * (D + 4) + c * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 kk = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * (D + 4) + c * 4);
#pragma unroll
          for (int r = 0; r < kF32R; ++r)
            x[r][j] = fmaf(qq[r].x, kk.x, fmaf(qq[r].y, kk.y, fmaf(qq[r].z, kk.z, fmaf(qq[r].w, kk.w, x[r][j]))));
        }
      }
#pragma unroll
      for (int r = 0; r < kF32R; ++r) {
        const int pos = s.len - s.n + (row0 + kF32R * ty + r) / p.G;
        float mx = neg_inf();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = key0 + tx + 16 * j;
          const bool vis = t <= pos && t < s.len && (p.window <= 0 || t > pos - p.window);
          if (!vis) x[r][j] = neg_inf();
          mx = fmaxf(mx, x[r][j]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        // m in scaled log2 units (the scale is positive)
        const float mn = fmaxf(m[r], mx == neg_inf() ? mx : mx * p.scale_log2);
        const float ref = mn == neg_inf() ? 0.f : mn;
        const float a = m[r] == neg_inf() ? 0.f : exp2f(m[r] - mn);
        m[r] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = x[r][j] == neg_inf() ? 0.f : exp2f(fmaf(x[r][j], p.scale_log2, -ref));
          ps[(kF32R * ty + r) * (kF32Keys + 4) + tx + 16 * j] = e;
          sum += e;
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[r] = l[r] * a + sum;
#pragma unroll
        for (int c = 0; c < OC; ++c) {
          o[r][c].x *= a;
          o[r][c].y *= a;
          o[r][c].z *= a;
          o[r][c].w *= a;
        }
      }
      __syncwarp();  // a row's probabilities are written and read by the same half-warp
#pragma unroll 2
      for (int t = 0; t < kF32Keys; t += 2) {
        float2 pp[kF32R];
#pragma unroll
        for (int r = 0; r < kF32R; ++r) pp[r] = *reinterpret_cast<const float2*>(ps + (kF32R * ty + r) * (kF32Keys + 4) + t);
#pragma unroll
        for (int c = 0; c < OC; ++c) {
          const float4 v0 = *reinterpret_cast<const float4*>(vs + t * D + tx * 4 + 64 * c);
          const float4 v1 = *reinterpret_cast<const float4*>(vs + (t + 1) * D + tx * 4 + 64 * c);
#pragma unroll
          for (int r = 0; r < kF32R; ++r) {
            o[r][c].x = fmaf(pp[r].y, v1.x, fmaf(pp[r].x, v0.x, o[r][c].x));
            o[r][c].y = fmaf(pp[r].y, v1.y, fmaf(pp[r].x, v0.y, o[r][c].y));
            o[r][c].z = fmaf(pp[r].y, v1.z, fmaf(pp[r].x, v0.z, o[r][c].z));
            o[r][c].w = fmaf(pp[r].y, v1.w, fmaf(pp[r].x, v0.w, o[r][c].w));
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < kF32R; ++r) {
      const int mrow = kF32R * ty + r;
      if (slot >= 0 && tx == 0) p.part_ml[(int64_t)slot * kF32Rows + mrow] = make_float2(m[r], l[r]);
      const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
      if (mrow < rows)
#pragma unroll
        for (int c = 0; c < OC; ++c) store(mrow, tx * 4 + 64 * c, o[r][c], inv);
    }
  }
}

template <int D, bool LIGHT>
static cudaError_t launch_f32(const ServeAttnParams& p, cudaStream_t stream) {
  auto kern = chunk_attn_f32<D, LIGHT>;
  const size_t smem = f32_smem_bytes<D>();
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)smem);
  if (e != cudaSuccess) return e;
  if (p.first) {
    kern<<<p.grid, kF32Threads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  return launch_dependent(kern, dim3(p.grid), dim3(kF32Threads), smem, stream, 0u, p);
}

cudaError_t launch_chunk_f32(const ServeAttnParams& p, cudaStream_t stream) {
  if (p.light) return p.D == 128 ? launch_f32<128, true>(p, stream) : launch_f32<64, true>(p, stream);
  return p.D == 128 ? launch_f32<128, false>(p, stream) : launch_f32<64, false>(p, stream);
}

}  // namespace specv
