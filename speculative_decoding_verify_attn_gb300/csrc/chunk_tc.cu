// Chunk attention on the 5th-generation tensor core: bf16 chunks of more than kMmaMaxRows query rows
// per sequence and kv head over a paged cache, and packed prompts.
//
// One CTA per SM takes the pieces of the plan (chunk_plan.cu) in turn: 256 query rows (tokens x heads
// of one kv head's group, two blocks of 128) against 128-key tiles.  Flash attention with the scores
// of a tile in TMEM: S_w = Q_w K^T (M = N = 128, both operands in shared memory), then
// P_w = 2^(s * scale - mu) rounded to bf16 over S_w's first 64 columns, then O_w += P_w V (P from TMEM,
// V as an MN-major operand).  mu is the maximum of the piece's first tile; later tiles take no maximum
// but look at their row sums, and only a sum above 2^20 moves mu (O is then rescaled in TMEM and the
// tile done again).  Any mu gives the same normalised result as long as nothing overflows.
//   warps 0, 1    loaders: K and V tiles into a ring of 32 KB stages (D = 128).  A tile that lies
//                 wholly inside the sequence comes by TMA; edges (the sequence's end, tokens before the
//                 window, bad page ids) and pages too small for TMA by cp.async with zeros in the gaps,
//                 so nothing outside [lo, len) reaches the tensor core, NaN or not.
//   warp 3        relay of cp.async tiles to the tensor core.
//   warp 2        MMA issuer (one lane): P V of a tile and Q K^T of the next for block 0, then for block
//                 1.  One issuer, because products of two issuers interleave in the tensor pipe: both
//                 blocks' scores are then ready at the same time, and the blocks run in step instead
//                 of one block's probabilities under the other's products.  The lane is chosen by
//                 elect.sync: with lane == 0 the products of a tile took 3000 cycles to issue instead
//                 of the 2050 they take to run (16K prompt: 1.85 ms against 1.34).
//   warps 4-11    two warpgroups, a thread per query row.
// Why 128-key tiles: an operand in shared memory is read anew by every instruction; per pair of blocks
// and 128 keys that is 192 KB of reads with 128-key scores and 256 KB with 64-key ones, against 2048
// cycles of products at 128 B per cycle.
// Measured (32/8 heads of 128), from a cool GPU to one at its power cap: one 16K prompt 1.34-1.46 ms,
// 1.64-1.51 PFLOP/s, 84-78% of the measured matrix rate (without any softmax arithmetic 1.28 ms on the cool
// one); a 2048-token chunk at 32K 0.67-0.74 ms, 1.6-1.45 PFLOP/s; 16 packed prompts of 60-2000 tokens 0.20 ms,
// 0.90 PFLOP/s (a piece costs 7000 cycles beside its 128-key steps of 2600); 16 sequences of 64K-128K with 56
// rows 0.96-0.975 ms, 6.75-6.65 TB/s.
// TMEM columns (512): block w at 256 w: S [0, 128), P over [0, 64), O [128, 128 + D).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch_cache.h"
#include "serve_common.cuh"
#include "serve_internal.h"
#include "tcgen05.cuh"

namespace specv {

constexpr int kCtThreads = 128 + 2 * 128;
constexpr uint32_t kCtTmemCols = 512;
constexpr int kCtHalf = 128 * 128;  // 128 rows of one 64-column half: 16 KB
// A row's sum over one tile up to which its reference stays (P is then below it, far inside bf16's and
// fp32's range, and the final division removes the reference).
constexpr float kCtMaxSum = 1048576.f;

template <int D>
struct Ct {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kCtHalf;       // a K or V tile, or a Q block
  static constexpr int kStages = D == 128 ? 5 : 10;     // 160 KB
  static constexpr size_t kSmem = 1024 + 2 * (size_t)kTile + (size_t)kStages * kTile;
  static constexpr uint32_t kIdescQK = tc::idesc_bf16(128, 128, 0, 0);
  static constexpr uint32_t kIdescPV = tc::idesc_bf16(128, D, 0, 1);
};

__device__ __forceinline__ uint32_t ct_col_s(int w) { return 256u * w; }
__device__ __forceinline__ uint32_t ct_col_o(int w) { return 256u * w + 128u; }

// Units of the piece that block w's rows see: [b0, b1), empty for a block without rows.
__device__ __forceinline__ void ct_block_units(const ServeAttnParams& p, const PieceItem& it, int w, int& b0, int& b1) {
  const int rows = it.s.n * p.G, r0 = it.row0 + w * 128;
  b0 = b1 = it.u0;
  if (r0 >= rows) return;
  const int rl = min(r0 + 128, rows) - 1, base = it.s.len - it.s.n;
  const int first = p.window > 0 ? max(0, base + r0 / p.G + 1 - min(p.window, it.s.len)) : 0;
  b0 = max(it.u0, first / kTcKeys);
  b1 = max(b0, min(it.u1, (base + rl / p.G) / kTcKeys + 1));
}

template <int D, bool LIGHT>
__global__ void __launch_bounds__(kCtThreads, 1)
    chunk_attn_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ ServeAttnParams p) {
  using C = Ct<D>;
  constexpr int NS = C::kStages;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[NS], empty[NS], landed[NS];
  __shared__ uint64_t sfull[2], pfull[2], pvdone[2], ofree[2], qfull[2], drain;
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  __shared__ LightSeqs s_light;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* qs = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // [block][half][128 rows][128 B]
  uint8_t* stages = qs + 2 * C::kTile;
  const uint32_t qs_u32 = smem_u32(qs), stages_u32 = smem_u32(stages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 2);     // warp 0 (with the bytes of a TMA copy) and the relay
      mbar_init(&landed[i], 64);  // every loader thread, once its copies have landed
      mbar_init(&empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sfull[w], 1);
      mbar_init(&pfull[w], 4);
      mbar_init(&pvdone[w], 1);
      mbar_init(&ofree[w], 4);
      mbar_init(&qfull[w], 4);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) tc::alloc(&tmem_base, kCtTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait();  // the plan, and appended rows
  if (LIGHT) light_init(p, s_light);
  PieceList<LIGHT> list;
  list.init(p, &s_light);
  const int rounds = list.rounds;

  auto fail = [&]() {
    s_abort = 1;
    chunk_report<LIGHT>(p, (uint32_t)SPEC_STATUS_TIMEOUT);
  };

  // registers: 128 x 88 + 256 x 208 = 384 x 168, what the block was launched with
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");

  if (warp < 2) {
    // ------------------------------------------------------------------ loaders
    constexpr int CH = D / 8, RPI = 32 / CH;
    const __nv_bfloat16* kv[2] = {reinterpret_cast<const __nv_bfloat16*>(p.k),
                                  reinterpret_cast<const __nv_bfloat16*>(p.v)};
    int step = 0;
    bool ok = true;
    PieceRaw ahead = list.fetch(p, 0);
    for (int round = 0; ok && round < rounds; ++round) {
      const PieceItem it = piece_item(ahead);
      ahead = list.fetch(p, round + 1);
      for (int u = it.u0; ok && u < it.u1; ++u) {
        const int key0 = u * kTcKeys;
        // rows of the tile: offsets of this lane's two of the warp's 64 keys, -1 where zeros go
        bool tma = p.use_tma && key0 >= it.s.lo && key0 + kTcKeys <= it.s.len;
        int64_t off[2] = {-1, -1};
        int page = 0, in_page = 0;
        if (tma) {
          if (!p.paged) {
            in_page = it.s.q0 + key0;
          } else {
            const int t = key0 + (lane * p.tma_page_keys) % kTcKeys;
            page = __ldg(p.table + (int64_t)it.b * p.table_stride + t / p.page_size);
            in_page = t % p.page_size;
            tma = __all_sync(0xffffffffu, page >= 0 && page < p.num_pages);
          }
        }
        if (!tma) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = key0 + warp * 64 + i * 32 + lane;
            if (t >= it.s.lo && t < it.s.len) {
              off[i] = key_offset(p, it.s, it.b, it.g, t);
              if (off[i] < 0) chunk_report<LIGHT>(p, (uint32_t)SPEC_STATUS_BAD_PAGE);
            }
          }
        }
        const bool groups = !tma && (!p.paged || (p.page_size & 15) == 0) &&
                            __all_sync(0xffffffffu, off[0] >= 0 && off[1] >= 0);
#pragma unroll 1
        for (int x = 0; x < 2; ++x, ++step) {
          const int s = step % NS;
          const bool got = mbar_wait_spin(&empty[s], ((step / NS) & 1) ^ 1u, &s_abort);
          if (!__all_sync(0xffffffffu, got)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t dst = stages_u32 + s * C::kTile;
          if (tma) {
            if (warp == 0) {
              if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)C::kTile);
              __syncwarp();
              // whole tiles in one copy; pages below a tile in one copy per page and half
              const int n = p.tma_page_keys == kTcKeys ? 1 : kTcKeys / p.tma_page_keys * C::kHalves;
              const int src_lane = n == 1 ? 0 : lane / C::kHalves;
              const int pg = __shfl_sync(0xffffffffu, page, src_lane), ip = __shfl_sync(0xffffffffu, in_page, src_lane);
              if (lane < n) {
                const int half = n == 1 ? 0 : lane % C::kHalves;
                const uint32_t at = dst + half * kCtHalf + src_lane * p.tma_page_keys * 128;
                asm volatile(
                    "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
                    " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(at),
                    "l"(reinterpret_cast<uint64_t>(x == 0 ? &tmK : &tmV)), "r"(0), "r"(ip), "r"(half), "r"(it.g),
                    "r"(pg), "r"(smem_u32(&full[s]))
                    : "memory");
              }
            }
          } else if (groups) {
            // 16 consecutive tokens of one page at a time; for rows i * RPI + lane / CH the lane's part
            // of the place in the tile is constant, and i changes it by an offset and an XOR
            const int c = lane % CH, rl = lane / CH;
            const uint32_t at = dst + (c >> 3) * kCtHalf + (warp * 64 + rl) * 128 + (((c & 7) ^ rl) << 4);
            const int64_t step_b = p.kv_st * RPI;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __nv_bfloat16* src = kv[x] + __shfl_sync(0xffffffffu, off[q >> 1], (q & 1) * 16) + rl * p.kv_st + c * 8;
#pragma unroll
              for (int i = 0; i < 16 / RPI; ++i) {
                cp_async16((at + (q * 16 + i * RPI) * 128) ^ (((i * RPI) & 7) << 4), src);
                src += step_b;
              }
            }
          } else {
            const int c = lane % CH;
#pragma unroll 4
            for (int i = 0; i < 64 / RPI; ++i) {
              const int r = i * RPI + lane / CH;  // of the warp's 64 rows
              const int64_t o0 = __shfl_sync(0xffffffffu, off[0], r & 31), o1 = __shfl_sync(0xffffffffu, off[1], r & 31);
              const int64_t so = r < 32 ? o0 : o1;
              const int row = warp * 64 + r;
              cp_async16(dst + (c >> 3) * kCtHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                         kv[x] + (so < 0 ? 0 : so) + c * 8, so >= 0);
            }
          }
          if (tma) {
            mbar_arrive(&landed[s]);  // after warp 0 has announced the bytes
          } else {
            cp_async_track(&landed[s]);
            if (warp == 0 && lane == 0) mbar_arrive(&full[s]);
          }
        }
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    if (!ok || s_abort) {
      // copies still in flight into this CTA
      for (int i = 1; i <= min(step, NS); ++i) mbar_wait_spin(&full[(step - i) % NS], ((step - i) / NS) & 1, nullptr);
    }
  } else if (warp < 4) {
    if (warp == 3 && elect_one()) {
      // ---------------------------------------------------------------- relay: cp.async tiles that have landed
      // are made visible to the tensor core, which reads them through the async proxy, so that neither the
      // loaders nor the issuer wait for that
      int step = 0;
      bool ok = true;
      PieceRaw ahead = list.fetch(p, 0);
      for (int round = 0; ok && round < rounds; ++round) {
        const int steps = 2 * (ahead.a.w - ahead.a.z);
        ahead = list.fetch(p, round + 1);
        for (int i = 0; i < steps; ++i, ++step) {
          if (!mbar_wait_spin(&landed[step % NS], (step / NS) & 1, &s_abort)) {
            ok = false;
            break;
          }
          tc::fence_proxy_async_smem();
          mbar_arrive(&full[step % NS]);
        }
      }
      if (!ok) fail();
    }
    // ------------------------------------------------------------------ MMA issuer (warp 2, one lane)
    if (warp == 2 && elect_one()) {
      int step = 0, part[2] = {0, 0}, t[2] = {0, 0};  // pieces and tiles so far, by block
      bool ok = true;
      // S_w = Q_w K^T (behind P_w V of the tile before, whose P it overwrites)
      const uint32_t q_lo = tc::desc_lo(qs_u32, 16), k_lo = tc::desc_lo(stages_u32, 16);
      const uint32_t v_lo = tc::desc_lo(stages_u32, kCtHalf);
      auto issue_qk = [&](int w, int stage) {
        const uint32_t qa = q_lo + w * (C::kTile >> 4), kb = k_lo + stage * (C::kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t koff = ((ks >> 2) * kCtHalf + (ks & 3) * 32) >> 4;
          tc::mma_ss_lo(tmem + ct_col_s(w), qa + koff, kb + koff, C::kIdescQK, ks > 0 ? 1u : 0u);
        }
        tc::commit(&sfull[w]);
      };
      PieceRaw ahead = list.fetch(p, 0);
      for (int round = 0; ok && round < rounds; ++round) {
        const PieceItem it = piece_item(ahead);
        ahead = list.fetch(p, round + 1);
        if (it.u0 >= it.u1) continue;
        int b0[2], b1[2];
        ct_block_units(p, it, 0, b0[0], b1[0]);
        ct_block_units(p, it, 1, b0[1], b1[1]);
        for (int u = it.u0 - 1; u < it.u1; ++u) {  // V of unit u (none before the first), K of u + 1
          const int sv = step % NS, sk = (step + (u >= it.u0 ? 1 : 0)) % NS;
          if (u >= it.u0 && !mbar_wait_spin(&full[sv], (step / NS) & 1, &s_abort)) { ok = false; break; }
          if (u >= it.u0) ++step;
          const bool more = u + 1 < it.u1;
          if (more && !mbar_wait_spin(&full[sk], (step / NS) & 1, &s_abort)) { ok = false; break; }
          if (more) ++step;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (!ok) break;
            if (u >= b0[w] && u < b1[w]) {  // O_w += P_w V
              if ((u == b0[w] && part[w] >= 1 && !mbar_wait_spin(&ofree[w], (part[w] - 1) & 1, &s_abort)) ||
                  !mbar_wait_spin(&pfull[w], t[w] & 1, &s_abort)) {
                ok = false;
                break;
              }
              tc::fence_after();
              const uint32_t vb = v_lo + sv * (C::kTile >> 4);
#pragma unroll
              for (int ks = 0; ks < kTcKeys / 16; ++ks)
                tc::mma_ts_lo(tmem + ct_col_o(w), tmem + ct_col_s(w) + ks * 8, vb + ks * (2048 >> 4), C::kIdescPV,
                              (ks > 0 || u > b0[w]) ? 1u : 0u);
              if (u == b1[w] - 1) tc::commit(&pvdone[w]);
              ++t[w];
            }
            if (more && u + 1 >= b0[w] && u + 1 < b1[w]) {
              if (u + 1 == b0[w] && !mbar_wait_spin(&qfull[w], part[w] & 1, &s_abort)) {
                ok = false;
                break;
              }
              tc::fence_after();
              issue_qk(w, sk);
            }
          }
          if (!ok) break;
          if (u >= it.u0) tc::commit(&empty[sv]);
          if (more) tc::commit(&empty[sk]);
        }
        if (b1[0] > b0[0]) ++part[0];
        if (b1[1] > b0[1]) ++part[1];
      }
      if (!ok) {
        fail();
        tc::commit(&drain);  // every MMA issued so far has finished before TMEM is released
        mbar_wait_spin(&drain, 0, nullptr);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warpgroups
    const int w = (warp - 4) >> 2;
    const int sub = warp & 3;        // TMEM sub-partition of this warp
    const int m = sub * 32 + lane;   // TMEM lane = row of the block
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
    const uint32_t sbuf = tl + ct_col_s(w), obuf = tl + ct_col_o(w);
    const uint32_t qblock_u32 = qs_u32 + w * C::kTile;
    const float sc = p.scale_log2;

    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool got = mbar_wait_spin(bar, parity, &s_abort);
      return __all_sync(0xffffffffu, got);
    };
    // the next piece in which this block has tiles; pieces without leave an empty record
    int round = 0;
    PieceRaw ahead = list.fetch(p, 0);
    auto next_piece = [&](PieceItem& n, int& nb0, int& nb1) -> bool {
      while (round < rounds) {
        n = piece_item(ahead);
        ahead = list.fetch(p, ++round);
        ct_block_units(p, n, w, nb0, nb1);
        if (nb1 > nb0) return true;
        if (n.slot >= 0) p.part_ml[(int64_t)n.slot * kTcRows + w * 128 + m] = make_float2(neg_inf(), 0.f);
      }
      return false;
    };
    // the warp's 32 rows of a piece into shared memory (K-major, 128-byte swizzle; zeros for padding
    // rows), asynchronously
    // (token and head of the thread's own row in `tok` and `head`, tok < 0 for padding)
    auto start_q = [&](const PieceItem& n, int& tok, int& head) {
      constexpr int CH = D / 8, RPI = 32 / CH;
      const int r = n.row0 + w * 128 + m;
      tok = r / p.G;
      head = n.g * p.G + r - tok * p.G;
      if (r >= n.s.n * p.G) tok = -1;
      const int64_t mine = tok >= 0 ? (int64_t)(n.s.q0 + tok) * p.q_st + (int64_t)head * p.q_sh : -1;
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int row = i * RPI + lane / CH;
        const int64_t off = __shfl_sync(0xffffffffu, mine, row);
        cp_async16(qblock_u32 + (c >> 3) * kCtHalf + (sub * 32 + row) * 128 + (((c & 7) ^ (row & 7)) << 4),
                   reinterpret_cast<const __nv_bfloat16*>(p.q) + (off < 0 ? 0 : off) + c * 8, off >= 0);
      }
      cp_async_commit();
    };
    auto finish_q = [&]() {
      cp_async_wait<0>();
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[w]);
    };

    PieceItem it;
    int b0 = 0, b1 = 0, tok = -1, head = 0;
    bool have = next_piece(it, b0, b1), ok = true;
    if (have) {
      start_q(it, tok, head);
      finish_q();
    }
    int t = 0, part = 0;
    while (have && ok) {
      PieceItem nx;
      int nb0 = 0, nb1 = 0, ntok = -1, nhead = 0;
      bool have_next = false, looked = false;
      const bool real = tok >= 0;
      // position of the row's token; padding rows see what the last row sees
      const int pos = it.s.len - it.s.n + (real ? tok : it.s.n - 1);
      const int wlo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      float m_run = neg_inf(), l = 0.f;
      for (int u = b0; u < b1; ++u, ++t) {
        if (u == b1 - 1 && !looked) have_next = next_piece(nx, nb0, nb1);
        if (!warp_wait(&sfull[w], t & 1)) { ok = false; break; }
        tc::fence_after();
        if (u == b1 - 1 && have_next) start_q(nx, ntok, nhead);  // the piece's last Q K^T has read its rows
        const int hi = pos - u * kTcKeys, lo = wlo - u * kTcKeys;  // visible columns [lo, hi]
        const bool edge = __any_sync(0xffffffffu, hi < kTcKeys - 1 || lo > 0);
        // P = 2^(s * scale - mu) against the present reference, as bf16 pairs; only where a row's sum
        // says that a score lies far above it (or nothing has been seen yet) is the tile's maximum
        // taken, O rescaled and the tile done again
        uint32_t pk[64];
        float sum;
        bool exact = u == b0;
        for (;;) {
          uint32_t s0[32], s1[32], s2[32], s3[32];
          tc::ld32(sbuf, s0);
          tc::ld32(sbuf + 32, s1);
          tc::ld32(sbuf + 64, s2);
          tc::ld32(sbuf + 96, s3);
          tc::ld_wait(s0);
          tc::ld_wait(s1);
          tc::ld_wait(s2);
          tc::ld_wait(s3);
          if (edge) {
            auto hide = [&](uint32_t(&v)[32], int c0) {
              const int h = hi - c0, l = lo - c0;  // visible [l, h]
              const uint32_t vis = (h >= 31 ? ~0u : h < 0 ? 0u : (2u << h) - 1u) & (l <= 0 ? ~0u : l > 31 ? 0u : ~0u << l);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = (vis >> e) & 1u ? v[e] : 0xff800000u;
            };
            hide(s0, 0);
            hide(s1, 32);
            hide(s2, 64);
            hide(s3, 96);
          }
          if (exact) {
            float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              mx[0] = fmax3(mx[0], __uint_as_float(s0[e]), __uint_as_float(s0[e + 1]));
              mx[1] = fmax3(mx[1], __uint_as_float(s1[e]), __uint_as_float(s1[e + 1]));
              mx[2] = fmax3(mx[2], __uint_as_float(s2[e]), __uint_as_float(s2[e + 1]));
              mx[3] = fmax3(mx[3], __uint_as_float(s3[e]), __uint_as_float(s3[e + 1]));
            }
            const float raw_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float m_new = raw_max == neg_inf() ? m_run : fmaxf(m_run, raw_max * sc);
            const float alpha = m_run == neg_inf() ? 0.f : ex2_approx(m_run - m_new);
            l *= alpha;
            m_run = m_new;
            if (u > b0) {
              // the P V before has completed: this tile's Q K^T, issued after it, has
              uint32_t v[32];
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                tc::ld32(obuf + c * 32, v);
                tc::ld_wait(v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                tc::st32(obuf + c * 32, v);
              }
              tc::st_wait();
            }
          }
          const float nmu = m_run == neg_inf() ? 0.f : -m_run;
          float sums[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          auto chunk = [&](const uint32_t(&v)[32], int c) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              fma2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), sc, nmu, x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              add2(sums[e & 6], sums[(e & 6) + 1], p0, p1);
              pk[c * 16 + e / 2] = pack_bf16(p0, p1);
            }
          };
          chunk(s0, 0);
          chunk(s1, 1);
          chunk(s2, 2);
          chunk(s3, 3);
          sum = ((sums[0] + sums[1]) + (sums[2] + sums[3])) + ((sums[4] + sums[5]) + (sums[6] + sums[7]));
          if (exact || !__any_sync(0xffffffffu, !(sum <= kCtMaxSum) || m_run == neg_inf())) break;
          exact = true;
        }
        l += sum;
        __syncwarp();
        tc::st32(sbuf, reinterpret_cast<uint32_t(&)[32]>(pk[0]));
        tc::st32(sbuf + 32, reinterpret_cast<uint32_t(&)[32]>(pk[32]));
        tc::st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[w]);
        if (!looked && u + 1 < b1) {  // while this tile's products run
          have_next = next_piece(nx, nb0, nb1);
          looked = true;
        }
      }
      if (!ok) break;
      if (have_next) finish_q();
      // ---- epilogue, once the piece's last P V is done; meanwhile where the row goes.
      // bf16 rows on 16-byte boundaries: four lanes turn their four rows' 64 bytes around, so that a
      // store covers 64 bytes of a row instead of 16
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int64_t off = real ? (int64_t)(it.s.q0 + tok) * p.o_st + (int64_t)head * p.o_sh : -1;
      const bool quads = p.o_bf16 && __all_sync(0xffffffffu, !real || ((reinterpret_cast<uintptr_t>(p.o) + off * 2) & 15u) == 0);
      int64_t quad_off[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) quad_off[i] = __shfl_sync(0xffffffffu, off, (lane & ~3) + i);
      if (!warp_wait(&pvdone[w], part & 1)) { ok = false; break; }
      ++part;
      tc::fence_after();
      if (it.slot >= 0) {
        const int64_t rec = it.slot;
        float* dst = p.part_o + rec * D * kTcRows + w * 128 + m;
        uint32_t v[32];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          __syncwarp();
          tc::ld32(obuf + c * 32, v);
          tc::ld_wait(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) dst[(c * 32 + e) * kTcRows] = __uint_as_float(v[e]);
        }
        p.part_ml[rec * kTcRows + w * 128 + m] = make_float2(m_run, l);
      } else {
        // not unrolled: this code runs once per piece and its instructions come from far; 32 columns'
        // worth of them, fetched once, halve the time of four times as many
        uint32_t v[32];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          __syncwarp();
          tc::ld32(obuf + c * 32, v);
          tc::ld_wait(v);
          if (quads) {
            uint32_t x[4][4];  // [8 columns][pair]
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              x[e >> 3][(e >> 1) & 3] = pack_bf16(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv);
            // 4 x 4 transposition of 16-byte blocks over the quad: exchange with lanes ^ 1, then ^ 2
#pragma unroll
            for (int s = 1; s <= 2; s <<= 1) {
              const bool up = (lane & s) != 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i & s) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t give = up ? x[i][e] : x[i | s][e];
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, s);
                  if (up) x[i][e] = got;
                  else x[i | s][e] = got;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (quad_off[i] >= 0)
                *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + quad_off[i] + c * 32 + (lane & 3) * 8) =
                    make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
          } else if (real) {
            if (p.o_bf16) {
              __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + off + c * 32;
#pragma unroll
              for (int e = 0; e < 32; ++e) dst[e] = __float2bfloat16_rn(__uint_as_float(v[e]) * inv);
            } else {
              float* dst = reinterpret_cast<float*>(p.o) + off + c * 32;
              if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<float4*>(dst + e) =
                      make_float4(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv,
                                  __uint_as_float(v[e + 2]) * inv, __uint_as_float(v[e + 3]) * inv);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) dst[e] = __uint_as_float(v[e]) * inv;
              }
            }
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ofree[w]);
      have = have_next;
      it = nx;
      b0 = nb0;
      b1 = nb1;
      tok = ntok;
      head = nhead;
    }
    if (!ok) fail();
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 2) {
    __syncwarp();
    tc::fence_after();
    tc::dealloc(tmem, kCtTmemCols);
  }
}

template <int D, bool LIGHT>
static cudaError_t launch_tc(const ServeAttnParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                             cudaStream_t stream) {
  auto kern = chunk_attn_tc<D, LIGHT>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), (int)Ct<D>::kSmem);
  if (e != cudaSuccess) return e;
  if (p.first) {
    kern<<<p.grid, kCtThreads, Ct<D>::kSmem, stream>>>(*tmK, *tmV, p);
    return cudaGetLastError();
  }
  return launch_dependent(kern, dim3(p.grid), dim3(kCtThreads), Ct<D>::kSmem, stream, 0u, *tmK, *tmV, p);
}

cudaError_t launch_chunk_tc(const ServeAttnParams& p, const CUtensorMap* tmK, const CUtensorMap* tmV,
                            cudaStream_t stream) {
  if (p.light) return p.D == 128 ? launch_tc<128, true>(p, tmK, tmV, stream) : launch_tc<64, true>(p, tmK, tmV, stream);
  return p.D == 128 ? launch_tc<128, false>(p, tmK, tmV, stream) : launch_tc<64, false>(p, tmK, tmV, stream);
}

}  // namespace specv
