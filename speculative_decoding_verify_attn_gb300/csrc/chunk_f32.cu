// Chunk attention on the CUDA cores: the fp32 form of the paged and packed operators.
//
// A CTA takes the pieces of the plan in turn: 32 query rows against 64-key tiles.  Thread (ty, tx)
// of 16 x 16 holds the scores of rows 2 ty, 2 ty + 1 and keys tx + 16 j, and the output columns
// 4 tx + 64 j of those rows.  fp32 throughout: scores by fp32 FMA, 2^x of the fused difference
// s * scale - m (the rounding of m is the same for the whole row and cancels in the normalisation),
// running maximum, sum and output in fp32.  Tiles come by cp.async, one ahead.  Bound: the FMA pipes for long chunks (the tensor cores
// have no fp32 type), HBM for few rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_cache.h"
#include "serve_common.cuh"
#include "serve_internal.h"

namespace specv {

constexpr int kF32Threads = 256;

template <int D>
constexpr size_t f32_smem_bytes() {
  return sizeof(float) * (kF32Rows * (D + 4) + 2 * kF32Keys * (D + 4) + 2 * kF32Keys * D + kF32Rows * (kF32Keys + 4));
}

template <int D>
__global__ void __launch_bounds__(kF32Threads) chunk_attn_f32(const __grid_constant__ ServeAttnParams p) {
  pdl_launch_dependents();
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                                // [32][D + 4]
  float* ks2 = qs + kF32Rows * (D + 4);          // [2][64][D + 4]
  float* vs2 = ks2 + 2 * kF32Keys * (D + 4);     // [2][64][D]
  float* ps = vs2 + 2 * kF32Keys * D;            // [32][64 + 4]
  __shared__ int64_t s_off[2][kF32Keys];         // where the keys of a unit lie, -1: zeros
  constexpr int C4 = D / 4, OC = D / 64;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float* q = reinterpret_cast<const float*>(p.q);
  const float* k = reinterpret_cast<const float*>(p.k);
  const float* v = reinterpret_cast<const float*>(p.v);
  pdl_wait();  // the plan, and appended rows
  PieceList list;
  list.init(p);
  for (int round = 0; round < list.rounds; ++round) {
    const PieceItem it = piece_item(list.fetch(p, round));
    if (it.u0 >= it.u1) continue;
    const int b = it.b, g = it.g, row0 = it.row0, u0 = it.u0, u1 = it.u1, slot = it.slot;
    const SeqInfo s = it.s;
    const int rows = min(kF32Rows, s.n * p.G - row0);
    const int warp_row = (tid >> 5) * 4;  // the warp's first row
    __syncthreads();
    for (int i = tid; i < kF32Rows * C4; i += kF32Threads) {
      const int r = i / C4, c = i % C4;
      const float4 x = r < rows ? *reinterpret_cast<const float4*>(q + q_offset(p, s, g, row0 + r) + c * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(qs + r * (D + 4) + c * 4) = x;
    }
    float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};
    float4 o[2][OC];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < OC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    // unit u + 1 is on its way while unit u is computed; its keys were looked up a unit earlier still
    auto look_up = [&](int u) {
      if (u < u1 && tid < kF32Keys) {
        const int key = u * kF32Keys + tid;
        int64_t off = -1;
        if (key >= s.lo && key < s.len) {
          off = key_offset(p, s, b, g, key);
          if (off < 0) atomicOr(p.status, (uint32_t)SPEC_STATUS_BAD_PAGE);
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
    look_up(u0);
    __syncthreads();
    issue(u0);
    look_up(u0 + 1);
    for (int u = u0; u < u1; ++u) {
      const int key0 = u * kF32Keys;
      const float *ks = ks2 + (u & 1) * kF32Keys * (D + 4), *vs = vs2 + (u & 1) * kF32Keys * D;
      __syncthreads();  // unit u + 1 looked up; the buffers of unit u - 1 are free
      issue(u + 1);
      cp_async_wait<1>();
      __syncthreads();  // unit u has landed, its offsets are free
      look_up(u + 2);
      if (warp_row >= rows) continue;  // rows of padding only
      float x[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[r][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < C4; ++c) {
        const float4 q0 = *reinterpret_cast<const float4*>(qs + (2 * ty) * (D + 4) + c * 4);
        const float4 q1 = *reinterpret_cast<const float4*>(qs + (2 * ty + 1) * (D + 4) + c * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 kk = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * (D + 4) + c * 4);
          x[0][j] = fmaf(q0.x, kk.x, fmaf(q0.y, kk.y, fmaf(q0.z, kk.z, fmaf(q0.w, kk.w, x[0][j]))));
          x[1][j] = fmaf(q1.x, kk.x, fmaf(q1.y, kk.y, fmaf(q1.z, kk.z, fmaf(q1.w, kk.w, x[1][j]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int pos = s.len - s.n + (row0 + 2 * ty + r) / p.G;
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
        // m in scaled log2 units; scale > 0 keeps the order (a negative or zero scale is refused)
        const float mn = fmaxf(m[r], mx == neg_inf() ? mx : mx * p.scale_log2);
        const float ref = mn == neg_inf() ? 0.f : mn;
        const float a = m[r] == neg_inf() ? 0.f : exp2f(m[r] - mn);
        m[r] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = x[r][j] == neg_inf() ? 0.f : exp2f(fmaf(x[r][j], p.scale_log2, -ref));
          ps[(2 * ty + r) * (kF32Keys + 4) + tx + 16 * j] = e;
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
#pragma unroll 4
      for (int t = 0; t < kF32Keys; ++t) {
        const float p0 = ps[(2 * ty) * (kF32Keys + 4) + t], p1 = ps[(2 * ty + 1) * (kF32Keys + 4) + t];
#pragma unroll
        for (int c = 0; c < OC; ++c) {
          const float4 vv = *reinterpret_cast<const float4*>(vs + t * D + tx * 4 + 64 * c);
          o[0][c].x = fmaf(p0, vv.x, o[0][c].x);
          o[0][c].y = fmaf(p0, vv.y, o[0][c].y);
          o[0][c].z = fmaf(p0, vv.z, o[0][c].z);
          o[0][c].w = fmaf(p0, vv.w, o[0][c].w);
          o[1][c].x = fmaf(p1, vv.x, o[1][c].x);
          o[1][c].y = fmaf(p1, vv.y, o[1][c].y);
          o[1][c].z = fmaf(p1, vv.z, o[1][c].z);
          o[1][c].w = fmaf(p1, vv.w, o[1][c].w);
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int mrow = 2 * ty + r;
      if (slot >= 0) {
        const int64_t rec = slot;
        if (tx == 0) p.part_ml[rec * kF32Rows + mrow] = make_float2(m[r], l[r]);
        float* dst = p.part_o + rec * D * kF32Rows + mrow;
#pragma unroll
        for (int c = 0; c < OC; ++c) {
          dst[(tx * 4 + 64 * c) * kF32Rows] = o[r][c].x;
          dst[(tx * 4 + 64 * c + 1) * kF32Rows] = o[r][c].y;
          dst[(tx * 4 + 64 * c + 2) * kF32Rows] = o[r][c].z;
          dst[(tx * 4 + 64 * c + 3) * kF32Rows] = o[r][c].w;
        }
      } else if (mrow < rows) {
        const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
        const int64_t off = o_offset(p, s, g, row0 + mrow);
#pragma unroll
        for (int c = 0; c < OC; ++c) {
          const float out[4] = {o[r][c].x * inv, o[r][c].y * inv, o[r][c].z * inv, o[r][c].w * inv};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t at = off + tx * 4 + 64 * c + e;
            if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(out[e]);
            else reinterpret_cast<float*>(p.o)[at] = out[e];
          }
        }
      }
    }
  }
}

template <int D>
static cudaError_t launch_f32(const ServeAttnParams& p, cudaStream_t stream) {
  auto kern = chunk_attn_f32<D>;
  const size_t smem = f32_smem_bytes<D>();
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.grid), dim3(kF32Threads), smem, stream, 0u, p);
}

cudaError_t launch_chunk_f32(const ServeAttnParams& p, cudaStream_t stream) {
  return p.D == 128 ? launch_f32<128>(p, stream) : launch_f32<64>(p, stream);
}

}  // namespace specv
