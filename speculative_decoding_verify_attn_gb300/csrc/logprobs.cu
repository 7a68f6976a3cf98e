// Log probabilities of given tokens, the rows' entropies and their top alternatives, in one pass
// over the logits.
//
// With m the running maximum, s = sum e^(x - m) and w = sum (x - m) e^(x - m), a row needs
//     lse = m + log s,    log p(v) = x_v - m - log s,    H = log s - w / s,
// and (m, s, w) of two parts of a row join as s' = s a + ..., w' = (w + (m - m') s) a + ..., a =
// e^(m - m').  Every thread keeps its own (m, s, w) in fp32 over 16-byte vectors (a few hundred
// elements each), joined by a fixed tree, so results do not depend on scheduling.
//
// Top alternatives: an id's key is (order of its logit, lower id first) as one 64-bit number; each
// warp keeps its K best keys sorted over its lanes.  A batch of vectors is looked at one by one only
// if its maximum, which the softmax needs anyway, reaches the warp's K-th value or the CTA's best
// K-th value so far (shared), so the list costs about K log(n / K) insertions per warp.
//
// Bound: HBM, one read of the logits.  A row is one CTA when there are enough rows to fill the GPU,
// else kSliceTarget / N slices whose records a second kernel joins (launched as a programmatic
// dependent).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "serve_internal.h"
#include "spec_serve.h"

namespace specv {

constexpr int kLpWarps = 8;
constexpr int kLpThreads = kLpWarps * 32;
constexpr int kLpVecs = 4;            // 16-byte vectors per lane and batch
constexpr int kSliceTarget = 608;     // CTAs wanted (four per SM) before rows are no longer sliced
constexpr int kMinSlice = 4096;       // elements of a slice at least (one fp32 batch of a CTA)

struct Stat {
  float m, s, w;
};
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  const float ref = r.m == neg_inf() ? 0.f : r.m;
  const float da = fmaxf(a.m - ref, -256.f), db = fmaxf(b.m - ref, -256.f);  // e^-256 is 0 in fp32
  const float ea = ex2_approx(da * kLog2e), eb = ex2_approx(db * kLog2e);
  r.s = a.s * ea + b.s * eb;
  r.w = (a.w + da * a.s) * ea + (b.w + db * b.s) * eb;
  return r;
}
__device__ __forceinline__ Stat warp_stat(Stat v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat u;
    u.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    u.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    u.w = __shfl_xor_sync(0xffffffffu, v.w, o);
    // both lanes of a pair join in the same order, so every lane ends with the same bits
    v = (threadIdx.x & o) ? stat_join(u, v) : stat_join(v, u);
  }
  return v;
}

typedef unsigned long long Key;
__device__ __forceinline__ Key make_key(float x, uint32_t id) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 as 0: equal logits compare equal
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((Key)o << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// The K best keys seen, sorted descending over the lanes of a warp (0: none yet).
struct TopList {
  Key mine = 0, thr = 0;
  __device__ __forceinline__ void insert(Key nk, int K) {
    const int lane = threadIdx.x & 31;
    const int pos = __popc(__ballot_sync(0xffffffffu, mine > nk));
    const Key up = __shfl_up_sync(0xffffffffu, mine, 1);
    if (lane >= pos) mine = lane == pos ? nk : up;
    thr = __shfl_sync(0xffffffffu, mine, K - 1);
  }
  // all lanes offer one key each (0: none); those above `floor` and the K-th enter
  __device__ __forceinline__ void offer(Key k, Key floor, int K) {
    for (;;) {
      const unsigned hit = __ballot_sync(0xffffffffu, k > thr && k > floor);
      if (!hit) return;
      const int src = __ffs(hit) - 1;
      insert(__shfl_sync(0xffffffffu, k, src), K);
      if ((threadIdx.x & 31) == src) k = 0;
    }
  }
};

template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;
  uint4 v;
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = BF16 ? (&v.x)[e >> 1] : (&v.x)[e];
    if (!BF16) return __uint_as_float(w);
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <bool BF16>
__device__ __forceinline__ float load_elem(const void* row, int64_t i) {
  if (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[i]);
  return reinterpret_cast<const float*>(row)[i];
}

// What a row's joined statistics and sorted keys say (one warp).
__device__ __forceinline__ void write_row(const LogprobParams& p, int row, const Stat& t, Key mine, float given,
                                          int tok_state) {
  const int lane = threadIdx.x & 31;
  const bool none = t.m == neg_inf();  // nothing but -inf
  const float ls = none ? 0.f : logf(t.s);
  if (lane == 0) {
    if (p.logprobs) p.logprobs[row] = tok_state < 0 ? 0.f : (none ? neg_inf() : (given - t.m) - ls);
    if (p.entropy) p.entropy[row] = none ? 0.f : fmaxf(ls - t.w / t.s, 0.f);
  }
  if (lane < p.K) {
    p.top_ids[(int64_t)row * p.K + lane] = (int32_t)~(uint32_t)mine;
    p.top_lp[(int64_t)row * p.K + lane] = none ? neg_inf() : (key_value(mine) - t.m) - ls;
  }
}
// The given token's logit; state -1 for an id outside [0, V), 0 without tokens.
template <bool BF16>
__device__ __forceinline__ float given_logit(const LogprobParams& p, const void* row_ptr, int row, int& state) {
  state = 0;
  if (!p.tokens) return 0.f;
  const int t = p.tokens[row];
  if (t < 0 || t >= p.V) {
    state = -1;
    return 0.f;
  }
  return load_elem<BF16>(row_ptr, t);
}

template <bool BF16, bool TOP>
__global__ void __launch_bounds__(kLpThreads) logprob_stats(const __grid_constant__ LogprobParams p) {
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) status_clear_for_launch(p.status);
  __shared__ Key s_keys[kLpWarps][32];
  __shared__ Stat s_stat[kLpWarps];
  __shared__ Key s_floor;  // the best K-th key of the CTA's warps: lower keys are not among the K best
  constexpr int VN = Vec<BF16>::N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const char* row_ptr = reinterpret_cast<const char*>(p.logits) + (int64_t)row * p.stride * (BF16 ? 2 : 4);
  // 16-byte vectors of the row; up to VN - 1 elements before and after them go one by one
  const int head = min(p.V, (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(row_ptr) & 15u)) & 15u) / (BF16 ? 2 : 4)));
  const int nvec = (p.V - head) / VN;
  const uint4* body = reinterpret_cast<const uint4*>(row_ptr + (int64_t)head * (BF16 ? 2 : 4));
  const int per = (nvec + p.slices - 1) / p.slices;
  const int v0 = min(nvec, slice * per), v1 = min(nvec, v0 + per);
  if (TOP && threadIdx.x == 0) s_floor = 0;
  if (TOP) __syncthreads();

  Stat st{neg_inf(), 0.f, 0.f};
  TopList top;
  auto single = [&](int i, bool in) {  // one element per lane, outside the vectors
    const float x = in ? load_elem<BF16>(row_ptr, i) : neg_inf();
    if (in) st = stat_join(st, Stat{x, x == neg_inf() ? 0.f : 1.f, 0.f});
    if (TOP) top.offer(in ? make_key(x, (uint32_t)i) : 0, 0, p.K);
  };
  // a warp meets its ids in ascending order (the head here, the tail at the end)
  if (slice == 0 && warp == 0 && head > 0) single(lane, lane < head);

  constexpr int kStep = kLpWarps * 32 * kLpVecs;
  Vec<BF16> cur[kLpVecs], nxt[kLpVecs];
  const uint32_t ninf2 = BF16 ? 0xff80ff80u : 0xff800000u;
  auto fetch = [&](Vec<BF16>(&d)[kLpVecs], int base) {
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u) {
      const int i = base + u * 32 + lane;
      d[u].v = i < v1 ? __ldcs(body + i) : make_uint4(ninf2, ninf2, ninf2, ninf2);
    }
  };
  int base = v0 + warp * 32 * kLpVecs;
  if (base < v1) fetch(cur, base);
  for (; base < v1; base += kStep) {
    if (base + kStep < v1) fetch(nxt, base + kStep);
    float vm[kLpVecs], bm = neg_inf();
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u) {
      vm[u] = cur[u].get(0);
#pragma unroll
      for (int e = 1; e < VN; ++e) vm[u] = fmaxf(vm[u], cur[u].get(e));
      bm = fmaxf(bm, vm[u]);
    }
    if (bm > st.m) {
      const float d = fmaxf(st.m - bm, -256.f);
      const float a = ex2_approx(d * kLog2e);
      st.w = (st.w + d * st.s) * a;
      st.s *= a;
      st.m = bm;
    }
    const float ref = st.m == neg_inf() ? 0.f : st.m;
    float s2[2] = {0.f, 0.f}, w2[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u)
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        const float d = fmaxf(cur[u].get(e) - ref, -256.f);  // -inf: e^-256 is 0 in fp32
        const float x = ex2_approx(d * kLog2e);
        s2[e & 1] += x;
        w2[e & 1] = fmaf(d, x, w2[e & 1]);
      }
    st.s += s2[0] + s2[1];
    st.w += w2[0] + w2[1];
    if (TOP) {
      const Key floor = *reinterpret_cast<volatile Key*>(&s_floor);
      // within the warp later ids lose ties, so the K-th value must be exceeded; against the other
      // warps' floor a tie may still win
      const bool full = top.thr != 0;
      const float tf = key_value(top.thr), ff = floor ? key_value(floor) : neg_inf();
      if (__any_sync(0xffffffffu, (!full || bm > tf) && bm >= ff)) {
#pragma unroll
        for (int u = 0; u < kLpVecs; ++u) {
          const int i = base + u * 32 + lane;
          if (!__any_sync(0xffffffffu, (top.thr == 0 || vm[u] >= key_value(top.thr)) && vm[u] >= ff)) continue;
#pragma unroll
          for (int e = 0; e < VN; ++e)
            top.offer(i < v1 ? make_key(cur[u].get(e), (uint32_t)(head + i * VN + e)) : 0, floor, p.K);
        }
        if (lane == 0 && top.thr > floor) atomicMax(&s_floor, top.thr);
      }
    }
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u) cur[u] = nxt[u];
  }
  const int tail0 = head + nvec * VN;
  if (slice == p.slices - 1 && warp == 0 && tail0 < p.V) single(tail0 + lane, tail0 + lane < p.V);

  st = warp_stat(st);
  if (lane == 0) s_stat[warp] = st;
  if (TOP) s_keys[warp][lane] = top.mine;
  __syncthreads();
  if (warp != 0) return;
  st = s_stat[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) {
    st = stat_join(st, s_stat[w]);
    if (TOP) top.offer(lane < p.K ? s_keys[w][lane] : 0, 0, p.K);
  }
  if (p.slices == 1) {
    int state;
    const float given = given_logit<BF16>(p, row_ptr, row, state);
    if (state < 0 && lane == 0) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_TOKEN);
    write_row(p, row, st, top.mine, given, state);
  } else {
    if (lane == 0) p.part_stat[blockIdx.x] = make_float4(st.m, st.s, st.w, 0.f);
    if (TOP && lane < p.K) p.part_keys[(int64_t)blockIdx.x * p.K + lane] = top.mine;
  }
}

// Joins the slices of a row (one warp per row).
template <bool BF16>
__global__ void __launch_bounds__(32) logprob_join(const __grid_constant__ LogprobParams p) {
  const int row = blockIdx.x, lane = threadIdx.x;
  const char* row_ptr = reinterpret_cast<const char*>(p.logits) + (int64_t)row * p.stride * (BF16 ? 2 : 4);
  int state;
  const float given = given_logit<BF16>(p, row_ptr, row, state);
  pdl_wait();
  Stat st{neg_inf(), 0.f, 0.f};
  for (int i = lane; i < p.slices; i += 32) {
    const float4 v = __ldcg(p.part_stat + (int64_t)row * p.slices + i);
    st = stat_join(st, Stat{v.x, v.y, v.z});
  }
  st = warp_stat(st);
  TopList top;
  const int nk = p.slices * p.K;
  for (int i0 = 0; i0 < nk; i0 += 32) {
    const int i = i0 + lane;
    top.offer(i < nk ? __ldcg(p.part_keys + (int64_t)row * nk + i) : 0, 0, p.K);
  }
  if (state < 0 && lane == 0) atomicOr(p.status, (uint32_t)SPEC_STATUS_BAD_TOKEN);
  write_row(p, row, st, top.mine, given, state);
}

int logprob_slices(int N, int V) {
  const int want = (kSliceTarget + N - 1) / N, most = (V + kMinSlice - 1) / kMinSlice;
  const int s = want < most ? want : most;
  return s < 1 ? 1 : s;
}

size_t logprob_workspace_bytes(int N, int V, int K) {
  if (N == 0) return 256;
  const int s = logprob_slices(N, V);
  size_t n = 256;
  if (s > 1) n += (size_t)N * s * (sizeof(float4) + (size_t)K * sizeof(Key));
  return (n + 255) & ~(size_t)255;
}
void logprob_workspace_carve(void* ws, LogprobParams* p) {
  char* b = reinterpret_cast<char*>(ws);
  p->status = reinterpret_cast<uint32_t*>(b);
  p->part_stat = reinterpret_cast<float4*>(b + 256);
  p->part_keys = reinterpret_cast<Key*>(b + 256 + (size_t)p->N * p->slices * sizeof(float4));
}

cudaError_t launch_token_logprobs(const LogprobParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)p.N * (unsigned)p.slices;
  const bool top = p.K > 0;
  if (p.bf16) {
    if (top) logprob_stats<true, true><<<grid, kLpThreads, 0, stream>>>(p);
    else logprob_stats<true, false><<<grid, kLpThreads, 0, stream>>>(p);
  } else {
    if (top) logprob_stats<false, true><<<grid, kLpThreads, 0, stream>>>(p);
    else logprob_stats<false, false><<<grid, kLpThreads, 0, stream>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.slices == 1) return e;
  return p.bf16 ? launch_dependent(logprob_join<true>, dim3(p.N), dim3(32), 0, stream, 0u, p)
                : launch_dependent(logprob_join<false>, dim3(p.N), dim3(32), 0, stream, 0u, p);
}

}  // namespace specv
