// Page tables of a paged cache: sequences forked, freed and grown (page_fork), pages in use moved together
// (page_compact), and the copies of pages that follow from either (page_copy).
//
// The tables are a few thousand to a few million words; what they need is several passes, each over what
// the one before has settled.  One thread-block cluster of eight CTAs makes them in one launch, with
// the cluster's hardware barrier between passes: no flags in memory, no waiting loops, no launch per pass.
// Counts are whole numbers, so the order of the atomics does not show in the result; ids are given
// out by prefix sums in the order of rows and pages.  The state is read into the workspace before any
// of it is written, so a call may work in place; after a data error nothing is written at all.
//
// Pass 0   copy refs; clear what the passes count in
// Pass 1   per row: check, note what it becomes; entries given back and shared change the counts
// Pass 2   per row (every CTA alike): does it need a copy, how many pages; prefix sums.  Free pages by rank
// Pass 3   entries, lengths, the counts of copied and new pages; the list of copies
// Pass 4   counts out
//
// Measured: 8 rows 12 us, 128 rows of 130 pages 16 us, 8000 pages compacted 10 us (five barriers of about 1 us, and
// the trips to memory between them).  It is eight SMs whatever the size: 512 rows of 2048 pages 228 us if they stay
// (198 without the look at their pages' holders), 344 if they change places, 227 compacted.
//
// page_copy: bound by HBM (each moved byte read and written once); 16 KB pieces of (page, array) dealt to all
// SMs, four 16-byte loads in flight per thread.  Measured: 2.1 GB moved in 670 us (6.2 TB/s), 113 MB in 17 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>

#include "cache_internal.h"
#include "common.cuh"

namespace specv {

namespace cg = cooperative_groups;

constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kPageCluster = 8;
constexpr int kPageCols = 128;  // entries of a row that a warp takes at a time
constexpr int kPageRows = 4;    // rows of a thread: 4096 at most over a CTA

// What all passes know of their place.
struct PageGrid {
  int rank, thread, threads, warp, warps, lane;
  __device__ __forceinline__ PageGrid() {
    rank = (int)blockIdx.x;
    thread = rank * kPageThreads + (int)threadIdx.x;
    threads = kPageCluster * kPageThreads;
    warp = thread >> 5;
    warps = threads >> 5;
    lane = threadIdx.x & 31;
  }
};

// Exclusive prefix over the CTA's threads; `total` gets the sum.
__device__ __forceinline__ int block_prefix(int v, int* sm, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  int pre = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPageWarps; ++w) {
    const int s = sm[w];
    if (w < warp) pre += s;
    total += s;
  }
  return pre + x - v;
}

__device__ __forceinline__ uint32_t status_of(const PageParams& p) { return __ldcg(p.status); }

// The pages of [lo, hi) that are free, by warp: each warp takes a range of whole 32s.
__device__ __forceinline__ void warp_range(int lo, int hi, int warp, int& a, int& e) {
  const int per = (((hi - lo) + kPageWarps * 32 - 1) / (kPageWarps * 32)) * 32;
  a = min(hi, lo + warp * per);
  e = min(hi, a + per);
}

// ------------------------------------------------------------------ fork
// What a warp needs of a row for 128 of its entries, read from the call's inputs alone.
struct ForkItem {
  int b, c0, parent, held, before, kept, need, grow, last;
  uint32_t bad;                                 // data errors, the same for the warp
  int mine[kPageCols / 32], from[kPageCols / 32];  // entries: the row's own, those it takes over (0 where there are none)
  int holders[kPageCols / 32];                     // of the row's own, before the call
  // entries [give(), held) are given back, [0, kept) taken over unless they are the row's already
  __device__ __forceinline__ int give() const { return parent == b ? kept : 0; }
  __device__ __forceinline__ int take() const { return parent == b ? 0 : kept; }

  __device__ __forceinline__ void read(const PageParams& p, int64_t item, int chunks, int lane) {
    b = (int)(item / chunks);
    c0 = (int)(item % chunks) * kPageCols;
    parent = p.parent[b];
    held = p.held[b];
    grow = p.grow ? p.grow[b] : 0;
    bad = 0;
    if (held < 0 || held > p.cols) bad = SPEC_STATUS_BAD_KV_LEN;
    if (parent < -1 || parent >= p.B) bad |= SPEC_STATUS_BAD_RANGE;
    before = kept = need = 0;
    last = -1;
    if (!bad && parent >= 0) {
      before = p.kv_len[parent];
      const int theirs = p.held[parent];
      if (theirs < 0 || theirs > p.cols || before < 0 || (int64_t)before > (int64_t)theirs * p.page_size || grow < 0 ||
          (int64_t)before + grow > (int64_t)p.cols * p.page_size) {
        bad = SPEC_STATUS_BAD_KV_LEN;
        before = 0;
      } else {
        kept = (int)(((int64_t)before + p.page_size - 1) / p.page_size);
        need = (int)(((int64_t)before + grow + p.page_size - 1) / p.page_size);
      }
    }
    if (parent < 0) grow = 0;
    const int32_t* own = p.table + (int64_t)b * p.table_st;
    const int32_t* theirs = p.table + (int64_t)max(parent, 0) * p.table_st;
#pragma unroll
    for (int i = 0; i < kPageCols / 32; ++i) {
      const int c = c0 + i * 32 + lane;
      mine[i] = !bad && c < held ? own[c] : 0;
      from[i] = !bad && c < take() ? theirs[c] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPageCols / 32; ++i) holders[i] = mine[i] >= 0 && mine[i] < p.num_pages ? __ldg(p.refs + mine[i]) : 0;
    if (!bad && c0 == 0 && grow > 0 && before % p.page_size != 0) last = theirs[before / p.page_size];
  }
  // to the counts, and what the row becomes to `rows`
  __device__ __forceinline__ void apply(const PageParams& p, int lane) const {
    uint32_t wrong = bad;
    auto good = [&](int e) {
      if (e >= 0 && e < p.num_pages) return true;
      wrong = SPEC_STATUS_BAD_PAGE;
      return false;
    };
    if (!bad) {
#pragma unroll
      for (int i = 0; i < kPageCols / 32; ++i) {
        const int c = c0 + i * 32 + lane;
        if (c < held && good(mine[i])) {
          if (holders[i] <= 0) wrong = SPEC_STATUS_BAD_PAGE;  // it would go out again as a free page
          if (c >= give()) atomicSub(p.count + mine[i], 1);
        }
        if (c < take()) {
          if (good(from[i])) atomicAdd(p.count + from[i], 1);
          p.stage[(int64_t)b * p.cols + c] = from[i];
        }
      }
      if (c0 == 0 && lane == 0) {
        const bool writes = grow > 0 && before % p.page_size != 0;
        if (writes && good(last)) {
          atomicAdd(p.writers + last, 1);
          atomicMin(p.lowest + last, b);
        }
        int4* row = reinterpret_cast<int4*>(p.rows + b);
        row[0] = make_int4(parent, before, kept, need);
        row[1] = make_int4(last, writes, before + grow, 0);
      }
    }
    if (wrong) atomicOr(p.status, wrong);
  }
};

__global__ void __cluster_dims__(kPageCluster, 1, 1) __launch_bounds__(kPageThreads)
    page_fork(const __grid_constant__ PageParams p) {
  pdl_launch_dependents();
  __shared__ int s_sum[kPageWarps];
  __shared__ int s_free[kPageCluster];
  const cg::cluster_group cl = cg::this_cluster();
  const PageGrid at;
  const int tid = threadIdx.x;

  // ---- pass 0, and the reads of each warp's first item of pass 1
  const int chunks = (p.cols + kPageCols - 1) / kPageCols;
  const int64_t items = (int64_t)p.B * chunks;
  ForkItem x;
  if (at.warp < items) x.read(p, at.warp, chunks, at.lane);
  if (at.thread == 0) {
    *p.status = 0u;
    *p.n_pairs = 0;
  }
  for (int i = at.thread; i < p.num_pages; i += at.threads) {
    p.count[i] = __ldg(p.refs + i);
    p.writers[i] = 0;
    p.lowest[i] = INT_MAX;
  }
  cl.sync();

  // ---- pass 1: a warp per row and 128 entries
  for (int64_t item = at.warp; item < items; item += at.warps) {
    if (item != at.warp) x.read(p, item, chunks, at.lane);
    x.apply(p, at.lane);
  }
  cl.sync();
  if (status_of(p)) return;  // the same for all: nothing reports before the next barrier

  // ---- pass 2: every CTA goes through all rows; thread t takes rows t * per .. (so prefixes follow the rows)
  const int per = (p.B + kPageThreads - 1) / kPageThreads;
  int4 r0[kPageRows], r1[kPageRows];
#pragma unroll
  for (int i = 0; i < kPageRows; ++i) {
    const int b = tid * per + i;
    const int4* row = reinterpret_cast<const int4*>(p.rows + b);
    const bool in = i < per && b < p.B;
    r0[i] = in ? __ldcg(row) : make_int4(0, 0, 0, 0);
    r1[i] = in ? __ldcg(row + 1) : make_int4(0, 0, 0, 0);
  }
  // free pages (while the rows are on their way): counted by CTA, then listed by rank as far as they are needed
  const int range = (p.num_pages + kPageCluster - 1) / kPageCluster;
  const int lo = min(p.num_pages, at.rank * range), hi = min(p.num_pages, lo + range);
  int wa, we;
  warp_range(lo, hi, tid >> 5, wa, we);
  const uint32_t first_free = __ballot_sync(0xffffffffu, wa + at.lane < we && __ldcg(p.count + wa + at.lane) <= 0);
  int mine = 0;
#pragma unroll 4
  for (int i = wa + 32 + at.lane; i < we; i += 32) mine += __ldcg(p.count + i) <= 0;
  mine = __reduce_add_sync(0xffffffffu, mine) + __popc(first_free);
  int fresh = 0, copies = 0;
  bool copy[kPageRows];
#pragma unroll
  for (int i = 0; i < kPageRows; ++i) {
    copy[i] = false;
    if (r1[i].y) {
      const int holders = __ldcg(p.count + r1[i].x), writers = __ldcg(p.writers + r1[i].x), lowest = __ldcg(p.lowest + r1[i].x);
      copy[i] = holders > 1 && !(writers == holders && lowest == tid * per + i);
    }
    fresh += (int)copy[i] + r0[i].w - r0[i].z;
    copies += copy[i];
  }
  int need_all, copies_all;
  const int fresh0 = block_prefix(fresh, s_sum, need_all);
  const int copy0 = block_prefix(copies, s_sum, copies_all);
  __syncthreads();
  if (at.lane == 0) s_sum[tid >> 5] = mine;
  __syncthreads();
  int before_warp = 0, cta_free = 0;
#pragma unroll
  for (int w = 0; w < kPageWarps; ++w) {
    if (w < (tid >> 5)) before_warp += s_sum[w];
    cta_free += s_sum[w];
  }
  if (tid < kPageCluster) *cl.map_shared_rank(&s_free[at.rank], tid) = cta_free;
  cl.sync();
  int before_cta = 0, free_all = 0;
#pragma unroll
  for (int r = 0; r < kPageCluster; ++r) {
    if (r < at.rank) before_cta += s_free[r];
    free_all += s_free[r];
  }
  if (need_all > free_all) {  // the same for all CTAs
    if (at.thread == 0) atomicOr(p.status, (uint32_t)SPEC_STATUS_NO_PAGE);
    return;
  }
  int k = before_cta + before_warp;
  for (int i0 = wa; i0 < we && k < need_all; i0 += 32) {
    const int i = i0 + at.lane;
    const uint32_t m = i0 == wa ? first_free : __ballot_sync(0xffffffffu, i < we && __ldcg(p.count + i) <= 0);
    const int mine_at = k + __popc(m & ((1u << at.lane) - 1));
    if ((m >> at.lane & 1u) && mine_at < need_all) p.free_ids[mine_at] = i;
    k += __popc(m);
  }
  // what a row needs, where its pages begin in the list of free ones, and its place among the copies; by one CTA
  if (at.rank == 0) {
    int f = fresh0, c = copy0;
#pragma unroll
    for (int i = 0; i < kPageRows; ++i) {
      const int b = tid * per + i;
      if (i >= per || b >= p.B) continue;
      int4* row = reinterpret_cast<int4*>(p.rows + b);
      // parent, kept, need, first new page; page copied or -1, place of the copy, new length
      row[0] = make_int4(r0[i].x, r0[i].z, r0[i].w, f);
      row[1] = make_int4(copy[i] ? r1[i].x : -1, c, r1[i].z, 0);
      f += (int)copy[i] + r0[i].w - r0[i].z;
      c += copy[i];
    }
  }
  cl.sync();

  // ---- pass 3
  if (at.thread == 0) *p.n_pairs = copies_all;
  for (int64_t item = at.warp; item < (int64_t)p.B * chunks; item += at.warps) {
    const int b = (int)(item / chunks), c0 = (int)(item % chunks) * kPageCols;
    const int4 r0 = __ldcg(reinterpret_cast<const int4*>(p.rows + b)), r1 = __ldcg(reinterpret_cast<const int4*>(p.rows + b) + 1);
    const int parent = r0.x, kept = r0.y, need = r0.z, first = r0.w;
    const bool copy = r1.x >= 0;
    int32_t* out = p.table_out + (int64_t)b * p.table_out_st;
    const int32_t* from = parent == b ? p.table + (int64_t)b * p.table_st : p.stage + (int64_t)b * p.cols;
#pragma unroll
    for (int i = 0; i < kPageCols / 32; ++i) {
      const int c = c0 + i * 32 + at.lane;
      if (c >= need) continue;
      if (c >= kept || (copy && c == kept - 1)) {
        // the copy is the row's first new page
        const int e = __ldcg(p.free_ids + first + (c >= kept ? (int)copy + c - kept : 0));
        out[c] = e;
        p.count[e] = 1;
      } else if (parent != b || out != from) {
        out[c] = parent == b ? from[c] : __ldcg(from + c);
      }
    }
    if (c0 == 0 && at.lane == 0) {
      p.held_out[b] = need;
      p.kv_len_out[b] = r1.z;
      if (copy) {
        p.pairs[r1.y] = make_int2(r1.x, __ldcg(p.free_ids + first));
        atomicSub(p.count + r1.x, 1);
      }
    }
  }
  cl.sync();

  // ---- pass 4
  for (int i = at.thread; i < p.num_pages; i += at.threads) p.refs_out[i] = __ldcg(p.count + i);
}

// ------------------------------------------------------------------ compact
// Pass 1: check the tables, count the pages in use.  Pass 2: list gaps and tails by rank.  Pass 3: pair them.
// Pass 4: tables and counts out.
__global__ void __cluster_dims__(kPageCluster, 1, 1) __launch_bounds__(kPageThreads)
    page_compact(const __grid_constant__ PageParams p) {
  pdl_launch_dependents();
  __shared__ int s_sum[kPageWarps];
  __shared__ int s_part[kPageCluster];
  const cg::cluster_group cl = cg::this_cluster();
  const PageGrid at;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (at.thread == 0) {
    *p.status = 0u;
    *p.n_pairs = 0;
  }
  cl.sync();

  // ---- pass 1
  const int chunks = (p.cols + kPageCols - 1) / kPageCols;
  for (int64_t item = at.warp; item < (int64_t)p.B * chunks; item += at.warps) {
    const int b = (int)(item / chunks), c0 = (int)(item % chunks) * kPageCols;
    const int held = p.held[b];
    if (held < 0 || held > p.cols) {
      if (at.lane == 0) atomicOr(p.status, (uint32_t)SPEC_STATUS_BAD_KV_LEN);
      continue;
    }
#pragma unroll
    for (int i = 0; i < kPageCols / 32; ++i) {
      const int c = c0 + i * 32 + at.lane;
      if (c >= held) continue;
      const int e = p.table[(int64_t)b * p.table_st + c];
      if (e < 0 || e >= p.num_pages || p.refs[e] <= 0) atomicOr(p.status, (uint32_t)SPEC_STATUS_BAD_PAGE);
    }
  }
  const int range = (p.num_pages + kPageCluster - 1) / kPageCluster;
  const int lo = min(p.num_pages, at.rank * range), hi = min(p.num_pages, lo + range);
  int wa, we;
  warp_range(lo, hi, warp, wa, we);
  int used = 0;
#pragma unroll 4
  for (int i = wa + at.lane; i < we; i += 32) used += p.refs[i] > 0;
  used = __reduce_add_sync(0xffffffffu, used);
  if (at.lane == 0) s_sum[warp] = used;
  __syncthreads();
  int used_before = 0, used_cta = 0;
#pragma unroll
  for (int w = 0; w < kPageWarps; ++w) {
    if (w < warp) used_before += s_sum[w];
    used_cta += s_sum[w];
  }
  if (tid < kPageCluster) *cl.map_shared_rank(&s_part[at.rank], tid) = used_cta;
  cl.sync();
  if (status_of(p)) return;  // the same for all: nothing reports behind the barrier
  int live = 0;
#pragma unroll
  for (int r = 0; r < kPageCluster; ++r) {
    if (r < at.rank) used_before += s_part[r];
    live += s_part[r];
  }

  // ---- pass 2: page i in use: the rank of it among those at or past `live`; free page below: its rank
  int k = used_before;
  for (int i0 = wa; i0 < we; i0 += 32) {
    const int i = i0 + at.lane;
    const bool in = i < we, is_used = in && p.refs[i] > 0;
    const uint32_t m = __ballot_sync(0xffffffffu, is_used);
    const int before = k + __popc(m & ((1u << at.lane) - 1));  // pages in use below i
    if (in && !is_used && i < live) p.writers[i - before] = i;  // gap number i - before
    // tail number: it is the (live - before)-th from the end of those in use
    if (is_used && i >= live) p.lowest[live - 1 - before] = i;
    if (in) p.free_ids[i] = is_used ? i : -1;
    if (in && i == live) *p.n_pairs = live - before;  // free pages below `live`; none if it is past all pages
    k += __popc(m);
  }
  cl.sync();
  // ---- pass 3: as many gaps below `live` as tails; the r-th tail from the start is the last but r
  const int gaps = __ldcg(p.n_pairs);
  for (int r = at.thread; r < gaps; r += at.threads) {
    const int to = __ldcg(p.writers + r), from = __ldcg(p.lowest + gaps - 1 - r);
    p.pairs[r] = make_int2(from, to);
    p.free_ids[from] = to;
    p.count[r] = p.refs[from];
  }
  if (at.thread == 0 && p.num_live) *p.num_live = live;
  cl.sync();
  // ---- pass 4
  for (int64_t item = at.warp; item < (int64_t)p.B * chunks; item += at.warps) {
    const int b = (int)(item / chunks), c0 = (int)(item % chunks) * kPageCols;
    const int held = p.held[b];
#pragma unroll
    for (int i = 0; i < kPageCols / 32; ++i) {
      const int c = c0 + i * 32 + at.lane;
      if (c < held) p.table_out[(int64_t)b * p.table_out_st + c] = __ldcg(p.free_ids + p.table[(int64_t)b * p.table_st + c]);
    }
  }
  // a page in use below `live` keeps its count, a gap takes its new page's, the others are free
  for (int i = at.thread; i < p.num_pages; i += at.threads) {
    const int n = p.refs[i];
    if (i >= live) p.refs_out[i] = 0;
    else if (n > 0) p.refs_out[i] = n;
    if (p.moved_out) p.moved_out[i] = __ldcg(p.free_ids + i);
  }
  for (int r = at.thread; r < gaps; r += at.threads) p.refs_out[__ldcg(p.writers + r)] = __ldcg(p.count + r);
}

// ------------------------------------------------------------------ copies
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads)
    page_copy(const __grid_constant__ PageArrays a, const int32_t* n_pairs, const int2* pairs) {
  pdl_wait();
  const int pieces = a.pieces[a.n];
  const int64_t total = (int64_t)__ldcg(n_pairs) * pieces;
  for (int64_t x = blockIdx.x; x < total; x += gridDim.x) {
    const int pair = (int)(x / pieces), piece = (int)(x % pieces);
    int lo = 0, hi = a.n;  // the array that the piece lies in
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.pieces[mid] <= piece) lo = mid;
      else hi = mid;
    }
    const int2 move = __ldcg(pairs + pair);
    const int64_t begin = (int64_t)(piece - a.pieces[lo]) * kPagePiece;
    const int n = (int)min((int64_t)kPagePiece, a.bytes[lo] - begin);
    const char* src = a.base[lo] + (int64_t)move.x * a.stride[lo] + begin;
    char* dst = a.base[lo] + (int64_t)move.y * a.stride[lo] + begin;
    if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | (uintptr_t)n) & 15) == 0) {
      const uint4* s = reinterpret_cast<const uint4*>(src);
      uint4* d = reinterpret_cast<uint4*>(dst);
      const int m = n / 16;
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (threadIdx.x + i * kCopyThreads < m) v[i] = __ldcs(s + threadIdx.x + i * kCopyThreads);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (threadIdx.x + i * kCopyThreads < m) __stcs(d + threadIdx.x + i * kCopyThreads, v[i]);
    } else {
      for (int i = threadIdx.x; i < n; i += kCopyThreads) dst[i] = src[i];
    }
  }
}

// ------------------------------------------------------------------ workspace and launches
static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static void page_layout(int B, int cols, int num_pages, bool compact, size_t (&at)[9]) {
  const size_t pages = up256((size_t)num_pages * sizeof(int32_t));
  const size_t moves = compact ? (size_t)num_pages / 2 + 1 : (size_t)B;
  at[0] = 256;                                              // number of pairs
  at[1] = at[0] + 256;                                      // pairs
  at[2] = at[1] + up256(moves * sizeof(int2));              // count
  at[3] = at[2] + pages;                                    // writers
  at[4] = at[3] + pages;                                    // lowest
  at[5] = at[4] + pages;                                    // free ids
  at[6] = at[5] + pages;                                    // rows
  at[7] = at[6] + (compact ? 0 : up256((size_t)B * sizeof(PageRow)));
  at[8] = at[7] + (compact ? 0 : up256((size_t)B * cols * sizeof(int32_t)));
}
size_t page_workspace_bytes(int B, int cols, int num_pages, bool compact) {
  size_t at[9];
  page_layout(B, cols, num_pages, compact, at);
  return at[8];
}
void page_workspace_carve(void* ws, PageParams* p) {
  size_t at[9];
  page_layout(p->B, p->cols, p->num_pages, p->compact != 0, at);
  char* b = reinterpret_cast<char*>(ws);
  p->status = reinterpret_cast<uint32_t*>(b);
  p->n_pairs = reinterpret_cast<int32_t*>(b + at[0]);
  p->pairs = reinterpret_cast<int2*>(b + at[1]);
  p->count = reinterpret_cast<int32_t*>(b + at[2]);
  p->writers = reinterpret_cast<int32_t*>(b + at[3]);
  p->lowest = reinterpret_cast<int32_t*>(b + at[4]);
  p->free_ids = reinterpret_cast<int32_t*>(b + at[5]);
  p->rows = reinterpret_cast<PageRow*>(b + at[6]);
  p->stage = reinterpret_cast<int32_t*>(b + at[7]);
}
cudaError_t launch_page_fork(const PageParams& p, cudaStream_t stream) {
  page_fork<<<kPageCluster, kPageThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_page_compact(const PageParams& p, cudaStream_t stream) {
  page_compact<<<kPageCluster, kPageThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_page_copy(const PageParams& p, const PageArrays& a, int max_pairs, cudaStream_t stream) {
  // about six CTAs an SM; the number of pairs is known on the device only
  const int64_t want = (int64_t)max_pairs * a.pieces[a.n];
  const unsigned grid = (unsigned)(want < 960 ? want : 960);
  return launch_dependent(page_copy, dim3(grid), dim3(kCopyThreads), 0, stream, 0u, a, p.n_pairs, p.pairs);
}

}  // namespace specv
