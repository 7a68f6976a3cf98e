// Shared by the kernels of the 8-bit cache: e4m3 values in registers, and block exponents.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "cache_internal.h"
#include "common.cuh"
#include "serve_common.cuh"

namespace specv {

// Two e4m3 values (low byte first) as fp16, which holds them exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
  return d;
}
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  lo = e4m3x2_to_f16x2((uint16_t)v);
  hi = e4m3x2_to_f16x2((uint16_t)(v >> 16));
}
// Two floats as e4m3, to nearest even, +-448 beyond it, 0x7f for NaN; `lo` in the low byte.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)f32x2_to_e4m3x2(a, b) | (uint32_t)f32x2_to_e4m3x2(c, d) << 16;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}

// 2^x for whole x in [-126, 127].
__device__ __forceinline__ float exp2_whole(int x) { return __int_as_float((x + 127) << 23); }
__device__ __forceinline__ int clamp_exp(int byte) { return min(max(byte, kMinExpByte), kMaxExpByte); }
// The exponent byte that a block with this largest magnitude needs: amax = m 2^k with 1 <= m < 2, and
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int needed_exp(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int k = (int)(bits >> 23) - 127;
  return clamp_exp(k - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0) + 127);
}
__device__ __forceinline__ int block_of(const Kv8Params& p, int slot) {
  return p.block_shift >= 0 ? slot >> p.block_shift : slot / p.block;
}
// Page and slot of token t of sequence b; page < 0 where the table's id is out of range.
__device__ __forceinline__ void page_slot(const ServeAttnParams& p, int b, int t, int& page, int& slot) {
  const int col = page_of(p, t);
  page = __ldg(p.table + (int64_t)b * p.table_stride + col);
  if (page >= p.num_pages) page = -1;
  slot = t - col * p.page_size;
}

// Queries in fp16: scaled by the power of two that brings the largest value to [2^14, 2^15), so that only parts
// 2^29 below that lose bits.  `inverse` undoes the scale.
__device__ __forceinline__ float f16_scale(float amax, float& inverse) {
  const int k = (int)(__float_as_uint(amax) >> 23) - 127;  // amax in [2^k, 2^(k + 1))
  const int up = amax > 0.f ? min(14 - k, 100) : 0;
  inverse = exp2_whole(-up);
  return exp2_whole(up);
}
// What the scores of such queries are multiplied by, kept where a block's 2^64 leaves it finite.
__device__ __forceinline__ float q_factor(float inverse, float scale_log2) {
  return fminf(inverse * scale_log2, 4.611686018427388e18f);  // 2^62
}

// ---- the softmax's sum where V's scales lie far apart.  Probabilities carry V's scale, p' = 2^(s + ev - R), and the
// sum takes p' 2^-ev.  The p' of a key whose scale is 2^100 below another's can leave the range of floats although
// the key counts as much as the other.  Where V's scales lie within 2^-28 .. 2^28 that cannot be: a key whose weight is
// within 2^-30 of the largest has p' > 2^-(28 + 64 + 30), whatever the others' scales.  Elsewhere the sum takes 2^(s - R).
constexpr int kFarLow = 127 - 28, kFarHigh = 127 + 28;  // bytes below and above are far
// l 2^x with f = 2^x, which may be below the range of floats where the product is not.
__device__ __forceinline__ float scale_sum(float l, float x, float f) {
  const float h = ex2_approx(0.5f * x);
  return x > -100.f ? l * f : l * h * h;
}
// The power of two by which a record's sum and values are divided (and its reference raised), so that no weight
// 2^(R_i - R) leaves the range before its sum is multiplied in; 0 for the usual sums.
__device__ __forceinline__ int sum_shift(float l) {
  const int k = (int)(__float_as_uint(l) >> 23) - 127;
  return l > 0.f && (k > 40 || k < -40) ? min(max(k, -100), 100) : 0;
}

}  // namespace specv
