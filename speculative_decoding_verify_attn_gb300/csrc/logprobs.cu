// Log probabilities of given tokens, the rows' entropies and their top alternatives, in one pass
// over the logits.
//
// With m the running maximum, s = sum e^(x - m) and w = sum (x - m) e^(x - m), a row needs
//     lse = m + log s,    log p(v) = x_v - m - log s,    H = log s - w / s,
// and (m, s, w) of two parts of a row join as s' = s a + ..., w' = (w + (m - m') s) a + ..., a =
// e^(m - m').  Every thread keeps its own (m, s, w) in fp32 over 16-byte vectors (V / 128 elements where a
// row is one CTA, 1002 at 128256), joined by a fixed tree, so results do not depend on scheduling.
//
// Top alternatives: an id's key is (order of its logit, lower id first) as one 64-bit number; each
// warp keeps its K best keys sorted over its lanes.  A batch of vectors is looked at one by one only
// if its maximum, which the softmax needs anyway, reaches a floor that the CTA's warps share: the
// least of the warps' ceil(K / 4)-th best values, at or above which K ids exist.  The first floor comes
// from the lanes' maxima of the first batch, before anything is inserted, so a row of n ids costs
// about K log(n / 4096) insertions in all.
//
// Bound: HBM, one read of the logits (4096 rows of 128256 bf16 logits: 160 us, 6.6 TB/s), and with
// alternatives the issue of the insertions (5: 203 us, 20: 240 us; fp32 logits with 20: 340 us, 6.2 TB/s).
// Four warps per CTA rather than eight: fewer warps share a row's ids, so each one's list is better and
// less is inserted (20 alternatives 279 us with eight).  A row is one CTA when there are enough rows to
// fill the GPU, else kSliceTarget / N slices whose records a second kernel joins (launched as a
// programmatic dependent).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "serve_internal.h"
#include "spec_serve.h"

namespace specv {

constexpr int kLpWarps = 4;
constexpr int kLpThreads = kLpWarps * 32;
constexpr int kLpVecs = 4;            // 16-byte vectors per lane and batch
constexpr int kLpCtasPerSm = 8;
constexpr int kSliceTarget = 608;     // CTAs wanted before rows are no longer sliced
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
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 as 0: equal logits compare equal
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ Key make_key(float x, uint32_t id) { return ((Key)order_of(x) << 32) | (uint32_t)~id; }
__device__ __forceinline__ float key_value(Key k) { return order_value((uint32_t)(k >> 32)); }
constexpr uint32_t kOrderNegInf = 0x007fffffu;  // order_of(-inf): no id is below it

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
  // all lanes offer one key each (0: none); those above the K-th enter
  __device__ __forceinline__ void offer(Key k, int K) {
    for (;;) {
      const unsigned hit = __ballot_sync(0xffffffffu, k > thr);
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
  __device__ __forceinline__ float max() const {
    if (!BF16) return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3)));
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
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
__global__ void __launch_bounds__(kLpThreads, kLpCtasPerSm) logprob_stats(const __grid_constant__ LogprobParams p) {
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) status_clear_for_launch(p.status);
  __shared__ Key s_keys[kLpWarps][32], s_top[32];
  __shared__ Stat s_stat[kLpWarps];
  __shared__ uint32_t s_rank[kLpWarps];  // order of each warp's ceil(K / 4)-th best value (or below it)
  __shared__ uint32_t s_floor;
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
  const int rank = (p.K + kLpWarps - 1) / kLpWarps;

  Stat st{neg_inf(), 0.f, 0.f};
  TopList top;
  auto single = [&](int i, bool in) {  // one element per lane, outside the vectors
    const float x = in ? load_elem<BF16>(row_ptr, i) : neg_inf();
    if (in) st = stat_join(st, Stat{x, x == neg_inf() ? 0.f : 1.f, 0.f});
    if (TOP) top.offer(in ? make_key(x, (uint32_t)i) : 0, p.K);
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
  fetch(cur, base);
  if (TOP) {
    // the first floor: the least of the warps' rank-th largest lane maxima
    float x = cur[0].max();
#pragma unroll
    for (int u = 1; u < kLpVecs; ++u) x = fmaxf(x, cur[u].max());
    uint32_t o = order_of(x), best = kOrderNegInf;
    for (int i = 0; i < rank; ++i) {
      best = __reduce_max_sync(0xffffffffu, o);
      const unsigned who = __ballot_sync(0xffffffffu, o == best);
      if (lane == __ffs(who) - 1) o = 0;
    }
    best = max(best, kOrderNegInf);
    if (lane == 0) s_rank[warp] = best;
    __syncthreads();
    const uint32_t f = __reduce_min_sync(0xffffffffu, s_rank[lane % kLpWarps]);
    if (threadIdx.x == 0) s_floor = f;
    __syncthreads();
  }
  for (; base < v1; base += kStep) {
    fetch(nxt, base + kStep);
    float bm = cur[0].max();
#pragma unroll
    for (int u = 1; u < kLpVecs; ++u) bm = fmaxf(bm, cur[u].max());
    if (bm > st.m) {
      const float d = fmaxf(st.m - bm, -256.f);
      const float a = ex2_approx(d * kLog2e);
      st.w = (st.w + d * st.s) * a;
      st.s *= a;
      st.m = bm;
    }
    const float nref = st.m == neg_inf() ? 0.f : -st.m;
    float s0 = 0.f, s1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u)
#pragma unroll
      for (int i = 0; i < VN / 2; ++i) {
        float d0 = cur[u].get(2 * i), d1 = cur[u].get(2 * i + 1), t0, t1;
        add2(d0, d1, nref, nref);
        d0 = fmaxf(d0, -256.f);  // -inf, and differences past fp32: e^-256 is 0 in fp32
        d1 = fmaxf(d1, -256.f);
        mul2(d0, d1, kLog2e, t0, t1);
        const float e0 = ex2_approx(t0), e1 = ex2_approx(t1);
        add2(s0, s1, e0, e1);
        fma2_acc(w0, w1, d0, d1, e0, e1);
      }
    st.s += s0 + s1;
    st.w += w0 + w1;
    if (TOP) {
      // a value counts from the floor on; within the warp, where later ids lose ties, from above the
      // K-th value on
      const uint32_t lim = max(*reinterpret_cast<volatile uint32_t*>(&s_floor), top.thr ? (uint32_t)(top.thr >> 32) + 1u : 0u);
      const float lf = order_value(lim);
      if (__any_sync(0xffffffffu, bm >= lf)) {
#pragma unroll
        for (int u = 0; u < kLpVecs; ++u) {
          if (!__any_sync(0xffffffffu, cur[u].max() >= lf)) continue;
          const int i = base + u * 32 + lane;
          uint32_t todo = 0;  // this lane's elements that count
#pragma unroll
          for (int e = 0; e < VN; ++e) todo |= cur[u].get(e) >= lf ? 1u << e : 0u;
          if (i >= v1) todo = 0;
          while (__any_sync(0xffffffffu, todo != 0)) {
            Key k = 0;
            if (todo) {
              const int e = __ffs(todo) - 1, word = BF16 ? e >> 1 : e;
              const uint32_t lo = (word & 1) ? cur[u].v.y : cur[u].v.x, hi = (word & 1) ? cur[u].v.w : cur[u].v.z;
              const uint32_t w = (word & 2) ? hi : lo;
              const float x = __uint_as_float(!BF16 ? w : (e & 1) ? (w & 0xffff0000u) : (w << 16));
              k = make_key(x, (uint32_t)(head + i * VN + e));
              todo &= todo - 1;
            }
            top.offer(k, p.K);
          }
        }
        // a better floor
        const uint32_t o = (uint32_t)(__shfl_sync(0xffffffffu, top.mine, rank - 1) >> 32);
        const uint32_t old = *reinterpret_cast<volatile uint32_t*>(&s_rank[warp]);
        __syncwarp();
        if (o > old) {
          if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&s_rank[warp]) = o;
          __syncwarp();
          const uint32_t f = __reduce_min_sync(0xffffffffu, reinterpret_cast<volatile uint32_t*>(s_rank)[lane % kLpWarps]);
          if (lane == 0) atomicMax(&s_floor, f);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kLpVecs; ++u) cur[u] = nxt[u];
  }
  const int tail0 = head + nvec * VN;
  if (slice == p.slices - 1 && warp == 0 && tail0 < p.V) single(tail0 + lane, tail0 + lane < p.V);

  st = warp_stat(st);
  if (lane == 0) s_stat[warp] = st;
  if (TOP) {
    // the warps' lists as one: a key's place is the number of greater keys; those below the floor
    // have no place among the K best
    s_keys[warp][lane] = lane < p.K && (uint32_t)(top.mine >> 32) >= *reinterpret_cast<volatile uint32_t*>(&s_floor) ? top.mine : 0;
    if (warp == 0) s_top[lane] = 0;
  }
  __syncthreads();
  if (TOP) {
    const Key mine = s_keys[warp][lane];
    // a list is sorted, so its first zero ends it
    int above = 0;
    for (int w = 0; w < kLpWarps; ++w)
      for (int i = 0; i < p.K; ++i) {
        const Key k = s_keys[w][i];
        if (k == 0) break;
        above += k > mine;
      }
    if (mine != 0 && above < p.K) s_top[above] = mine;
    __syncthreads();
  }
  if (warp != 0) return;
  st = s_stat[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) st = stat_join(st, s_stat[w]);
  const Key best = TOP ? s_top[lane] : 0;
  if (p.slices == 1) {
    int state;
    const float given = given_logit<BF16>(p, row_ptr, row, state);
    if (state < 0 && lane == 0) status_report(p.status, (uint32_t)SPEC_STATUS_BAD_TOKEN);
    write_row(p, row, st, best, given, state);
  } else {
    if (lane == 0) p.part_stat[blockIdx.x] = make_float4(st.m, st.s, st.w, 0.f);
    if (TOP && lane < p.K) p.part_keys[(int64_t)blockIdx.x * p.K + lane] = best;
  }
}

// Joins the slices of a row.  If there are more than K slices, the K-th of their best keys is a floor;
// at most K slices reach it, so at most K * K keys remain, whose places are counted out.
constexpr int kJoinThreads = 256;
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) logprob_join(const __grid_constant__ LogprobParams p) {
  __shared__ Key s_best[kSliceTarget];
  __shared__ Key s_cand[32 * 32];
  __shared__ Key s_top[32];
  __shared__ Key s_floor;
  __shared__ int s_n;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const char* row_ptr = reinterpret_cast<const char*>(p.logits) + (int64_t)row * p.stride * (BF16 ? 2 : 4);
  int state = 0;
  float given = 0.f;
  if (tid < 32) {
    given = given_logit<BF16>(p, row_ptr, row, state);
    s_top[lane] = 0;
    if (tid == 0) {
      s_floor = 1;
      s_n = 0;
    }
  }
  pdl_wait();
  Stat st{neg_inf(), 0.f, 0.f};
  if (tid < 32) {
    for (int i = lane; i < p.slices; i += 32) {
      const float4 v = __ldcg(p.part_stat + (int64_t)row * p.slices + i);
      st = stat_join(st, Stat{v.x, v.y, v.z});
    }
    st = warp_stat(st);
  }
  if (p.K > 0) {
    const Key* keys = p.part_keys + (int64_t)row * p.slices * p.K;
    if (p.slices > p.K) {
      for (int i = tid; i < p.slices; i += kJoinThreads) s_best[i] = __ldcg(keys + i * p.K);
      __syncthreads();
      for (int i = tid; i < p.slices; i += kJoinThreads) {
        const Key mine = s_best[i];
        int above = 0;
        for (int j = 0; j < p.slices; ++j) above += s_best[j] > mine;
        if (mine != 0 && above == p.K - 1) s_floor = mine;
      }
    }
    __syncthreads();
    for (int i = tid; i < p.slices * p.K; i += kJoinThreads) {
      const Key k = __ldcg(keys + i);
      if (k >= s_floor) s_cand[atomicAdd(&s_n, 1)] = k;
    }
    __syncthreads();
    for (int i = tid; i < s_n; i += kJoinThreads) {
      const Key mine = s_cand[i];
      int above = 0;
      for (int j = 0; j < s_n; ++j) above += s_cand[j] > mine;
      if (above < p.K) s_top[above] = mine;
    }
    __syncthreads();
  }
  if (tid >= 32) return;
  if (state < 0 && lane == 0) atomicOr(p.status, (uint32_t)SPEC_STATUS_BAD_TOKEN);
  write_row(p, row, st, s_top[lane], given, state);
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
  return p.bf16 ? launch_dependent(logprob_join<true>, dim3(p.N), dim3(kJoinThreads), 0, stream, 0u, p)
                : launch_dependent(logprob_join<false>, dim3(p.N), dim3(kJoinThreads), 0, stream, 0u, p);
}

}  // namespace specv
