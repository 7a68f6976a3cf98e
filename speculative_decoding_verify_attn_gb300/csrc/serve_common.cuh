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
// This thread's arrival on `bar`, made once its copies so far have landed.
__device__ __forceinline__ void cp_async_track(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
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
__device__ __forceinline__ int chunk_tiles(const ServeAttnParams& p, const SeqInfo& s) {
  return s.len > 0 ? (int)(((int64_t)s.n * p.G + p.row_tile - 1) / p.row_tile) : 0;
}
// The key units [u0, u1) that the rows of a tile see, row0 its first, in a chunk of n tokens over len keys.
__device__ __forceinline__ void tile_units(const ServeAttnParams& p, int n, int len, int row0, int& u0, int& u1) {
  const int base = len - n, last = min(n * p.G, row0 + p.row_tile) - 1;
  const int first_key = p.window > 0 ? max(0, base + row0 / p.G + 1 - min(p.window, len)) : 0;
  u0 = first_key / p.unit_keys;
  u1 = (base + last / p.G) / p.unit_keys + 1;
}
__device__ __forceinline__ int first_key_of(const ServeAttnParams& p, int n, int len) {
  return p.window > 0 ? max(0, len - n + 1 - min(p.window, len)) : 0;
}
// An attention kernel's report: in the call's first kernel only after this launch's clear.
template <bool LIGHT>
__device__ __forceinline__ void chunk_report(const ServeAttnParams& p, uint32_t bits) {
  if (LIGHT && p.first) status_report(p.status, bits);
  else atomicOr(p.status, bits);
}

// A light call's sequences, in shared memory: tiles before each, and its numbers.
struct LightSeqs {
  int pre[kLightMaxB + 1], q0[kLightMaxB], n[kLightMaxB], len[kLightMaxB];
};
// Whole CTA, after the grid-dependency wait: reads the sequences, clears the status where this kernel is
// the call's first, reports bad sequences and zeros the rows of a bad kv_len.
__device__ __forceinline__ void light_init(const ServeAttnParams& p, LightSeqs& l) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (p.first && blockIdx.x == 0 && tid == 0) status_clear_for_launch(p.status);
  if (tid < 32) {
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int n = 0;
      if (b < p.B) {
        const SeqInfo s = seq_info(p, b);
        n = chunk_tiles(p, s);
        l.q0[b] = s.q0;
        l.n[b] = s.n;
        l.len[b] = s.len;
        if (p.first && blockIdx.x == 0 && s.bad) status_report(p.status, s.bad);
      }
      int x = n;  // at most 2^22 each
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < p.B) l.pre[b] = run + x - n;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) l.pre[p.B] = run;
  }
  __syncthreads();
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (l.len[b] > 0 || l.n[b] == 0) continue;
    for (int64_t i = tid; i < (int64_t)l.n[b] * p.Hq * p.D; i += blockDim.x) {
      const int64_t r = i / p.D;
      const int64_t off = (l.q0[b] + r / p.Hq) * p.o_st + (r % p.Hq) * p.o_sh + i % p.D;
      if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[off] = __float2bfloat16_rn(0.f);
      else reinterpret_cast<float*>(p.o)[off] = 0.f;
    }
  }
}
struct PieceItem {
  int b, g, row0, u0, u1, slot;
  SeqInfo s;
};
// A piece as it lies in memory (u0 == u1: none, and no record).  Readers fetch a piece ahead.
struct PieceRaw {
  int4 a, b, c;
};
// The pieces of a CTA: first its share of the cut tiles, then small tiles (sorted by size, dealt forth
// and back over the CTAs from small_first on).
template <bool LIGHT>
struct PieceList {
  int n_big, n_small, first, ctas, rounds;
  const LightSeqs* light;
  __device__ __forceinline__ void init(const ServeAttnParams& p, const LightSeqs* seqs) {
    light = seqs;
    if (LIGHT) {
      n_big = first = 0;
      ctas = (int)gridDim.x;
      n_small = light->pre[p.B];  // tiles; pieces are that times Hkv
      rounds = (int)(((int64_t)n_small * p.Hkv + ctas - 1) / ctas);
      return;
    }
    const int4 h = __ldcg(reinterpret_cast<const int4*>(p.plan));
    n_big = (int)blockIdx.x < h.z ? __ldcg(p.big_count + blockIdx.x) : 0;
    n_small = h.x * p.Hkv;
    first = h.w;
    ctas = (int)gridDim.x - first;
    rounds = n_big + ((int)blockIdx.x >= first ? (n_small + ctas - 1) / ctas : 0);
  }
  __device__ __forceinline__ PieceRaw fetch(const ServeAttnParams& p, int round) const {
    PieceRaw r;
    r.a = r.c = make_int4(0, 0, 0, 0);
    r.b = make_int4(-1, 0, 0, 0);
    if (LIGHT) {
      const int64_t idx = (int64_t)round * ctas + blockIdx.x;
      if (idx < (int64_t)n_small * p.Hkv) {
        const int t = (int)(idx / p.Hkv);
        int lo = 0, hi = p.B;  // the last sequence that begins at tile t or before
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (light->pre[mid] <= t) lo = mid;
          else hi = mid;
        }
        const int n = light->n[lo], len = light->len[lo];
        r.a.x = lo;
        r.a.y = (t - light->pre[lo]) * p.row_tile;
        tile_units(p, n, len, r.a.y, r.a.z, r.a.w);
        r.b = make_int4(-1, light->q0[lo], n, len);
        r.c.x = first_key_of(p, n, len);
        r.c.y = (int)(idx - (int64_t)t * p.Hkv);
      }
    } else if (round < n_big) {
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
