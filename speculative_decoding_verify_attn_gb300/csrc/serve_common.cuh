// Shared by the attention kernels of the serving operators: what a sequence of the ragged batch is,
// where its rows and keys lie, and cp.async.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "serve_internal.h"
#include "spec_serve.h"

namespace specv {

// Sequence b of the batch: chunk rows q0 .. q0 + n - 1, `len` keys of which [lo, len) are seen by
// some row.  len == 0: no keys to attend to (n == 0, or bad data: `bad` holds the status flag; with
// n > 0 the rows' output is zero).
struct SeqInfo {
  int q0, n, len, lo;
  uint32_t bad;
};
__device__ __forceinline__ SeqInfo seq_info(const ServeAttnParams& p, int b) {
  SeqInfo s{0, 0, 0, 0, 0u};
  const int a = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
  if (a < 0 || e < a || e > p.T || e - a > p.max_q) {
    s.bad = (uint32_t)SPEC_STATUS_BAD_RANGE;
    return s;
  }
  s.q0 = a;
  s.n = e - a;
  if (s.n == 0) return s;
  const int len = p.kv_len ? __ldg(p.kv_len + b) : s.n;
  if (len < s.n || (p.paged && (int64_t)len > (int64_t)p.table_cols * p.page_size)) {
    s.bad = (uint32_t)SPEC_STATUS_BAD_KV_LEN;
    return s;
  }
  s.len = len;
  s.lo = p.window > 0 ? max(0, len - s.n + 1 - min(p.window, len)) : 0;
  return s;
}

// 16-byte asynchronous copy to shared memory; zeros instead when `valid` is false (nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ int page_of(const ServeAttnParams& p, int t) {
  return p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size;
}
// Element offset of token t's row of kv head g, or -1 for a page id out of range.
__device__ __forceinline__ int64_t key_offset(const ServeAttnParams& p, const SeqInfo& s, int b, int g, int t) {
  if (!p.paged) return (int64_t)(s.q0 + t) * p.kv_st + (int64_t)g * p.kv_sh;
  const int col = page_of(p, t);
  const int page = __ldg(p.table + (int64_t)b * p.table_stride + col);
  if (page < 0 || page >= p.num_pages) return -1;
  return (int64_t)page * p.kv_sp + (int64_t)(t - col * p.page_size) * p.kv_st + (int64_t)g * p.kv_sh;
}

// Element offset of chunk row r (token r / G of the chunk, head r % G of kv head g's group).
__device__ __forceinline__ int64_t q_offset(const ServeAttnParams& p, const SeqInfo& s, int g, int r) {
  return (int64_t)(s.q0 + r / p.G) * p.q_st + (int64_t)(g * p.G + r % p.G) * p.q_sh;
}
__device__ __forceinline__ int64_t o_offset(const ServeAttnParams& p, const SeqInfo& s, int g, int r) {
  return (int64_t)(s.q0 + r / p.G) * p.o_st + (int64_t)(g * p.G + r % p.G) * p.o_sh;
}

// ------------------------------------------------------------------ pieces of the chunk kernels
struct PieceItem {
  int b, g, row0, u0, u1, slot;
  SeqInfo s;
};
// A piece as it lies in memory (u0 == u1: none).  Readers fetch a piece ahead.
struct PieceRaw {
  int4 a, b, c;
};
// The pieces of a CTA: first its share of the cut tiles, then small tiles (sorted by size, dealt forth
// and back over the CTAs from small_first on).
struct PieceList {
  int n_big, n_small, first, ctas, rounds;
  __device__ __forceinline__ void init(const ServeAttnParams& p) {
    const int4 h = __ldcg(reinterpret_cast<const int4*>(p.plan));
    n_big = (int)blockIdx.x < h.z ? __ldcg(p.big_count + blockIdx.x) : 0;
    n_small = h.x * p.Hkv;
    first = h.w;
    ctas = (int)gridDim.x - first;
    rounds = n_big + ((int)blockIdx.x >= first ? (n_small + ctas - 1) / ctas : 0);
  }
  __device__ __forceinline__ PieceRaw fetch(const ServeAttnParams& p, int round) const {
    PieceRaw r;
    r.a = r.b = r.c = make_int4(0, 0, 0, 0);
    if (round < n_big) {
      const int4* src = reinterpret_cast<const int4*>(p.big + blockIdx.x * kBigPieces + round);
      r.a = __ldcg(src);
      r.b = __ldcg(src + 1);
      r.c = __ldcg(src + 2);
    } else if (round < rounds) {
      const int k = round - n_big, at = (int)blockIdx.x - first;
      const int64_t idx = (int64_t)k * ctas + ((k & 1) ? ctas - 1 - at : at);
      if (idx < n_small) {
        const int4* src = reinterpret_cast<const int4*>(p.items + idx / p.Hkv);
        r.a = __ldcg(src);
        r.b = __ldcg(src + 1);
        r.c.x = __ldcg(reinterpret_cast<const int*>(src + 2));
        r.c.y = (int)(idx % p.Hkv);
      }
    }
    return r;
  }
};
__device__ __forceinline__ PieceItem piece_item(const PieceRaw& r) {
  return PieceItem{r.a.x, r.c.y, r.a.y, r.a.z, r.a.w, r.b.x, SeqInfo{r.b.y, r.b.z, r.b.w, r.c.x, 0u}};
}

}  // namespace specv
