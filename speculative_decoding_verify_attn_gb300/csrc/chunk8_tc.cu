// Chunk attention on the 5th-generation tensor core over a cache in 8 bits: chunks of more than kMmaMaxRows query
// rows per sequence and kv head.  The pieces, the pipeline and the softmax are chunk_tc.cu's: 256 query rows (two
// blocks of 128) against 128-key tiles, S = Q K^T and O += P V with S, P and O in TMEM.  What differs:
//   The tensor core gets fp16: no kind takes a 16-bit and an 8-bit operand, and 8 bits are too few for queries
//   and probabilities.  fp16 holds e4m3 exactly and probabilities better than bf16.
//   warps 0-3, 5-7  loaders: groups of 32 keys of a K or V tile go to them in turn.  A thread reads 16 bytes of a
//                 key at a time and stores 32 bytes of fp16 where the tensor core wants them; the next group's page
//                 ids come meanwhile.  Values go through registers: raw rows in shared memory would add 512 cycles
//                 of its port to the 1536 that the products' operands take per 128 keys (810 us instead of 798).
//   warp 4        MMA issuer (one lane), as there.
//   warps 8-15    two warpgroups, a thread per query row.
// Scales: the 32 keys of a group are brought to their largest exponent by an exact fp16 product (nothing is done
// where they share one, as in blocks of 32 tokens or more); K's scale, V's exponent and its inverse scale go to
// the softmax through shared memory, four of each per tile.  There K's multiplies the scores of its 32
// columns, and V's is added to the exponent of the probabilities: p' = 2^(s + ev - mu), as in paged8_mma.cu;
// the sum of the softmax takes p' 2^-ev.  Keys more than 2^15 apart, which fp16 cannot bring together (a block of zeros
// has the least scale, one of a rolled back token may have a large one), keep their values as they are, and the softmax
// scales their scores one by one and counts them without V's scale, as it does where that is far from 1: in loops that the
// usual tile does not see (it takes 0.80 ms with the code of them and 0.79 without; a chunk with such keys in all tiles
// 1.4-1.7 ms).
// mu is 2^8 below the largest s + ev of the piece's first tile: 128 equal scores then stay below 2^15, a sum
// up to which fp16 holds every p', and steps of 2^-24 are 2^-32 of the largest.
// Query rows are scaled by powers of two into fp16, in place in shared memory, once per piece.
// Measured (32/8 heads of 128): a 2048-token chunk at 32K 0.80 ms, 1.34 PFLOP/s, 70% of the measured matrix rate.  128
// keys take 3500 cycles, 2050 of them products: the issuer waits 500 for tiles and 500 for probabilities, and its
// products run slower beside the loaders' stores.  24 sequences of 0-384 tokens, 16/4 heads of 64, 0.10 ms of 0.13.
// TMEM columns (512): block w at 256 w: S [0, 128), O [128, 128 + D), P over S's first 64 or, for rows of 64, in the last 64.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "cache_internal.h"
#include "common.cuh"
#include "kv8_common.cuh"
#include "launch_cache.h"
#include "serve_common.cuh"
#include "serve_internal.h"
#include "tcgen05.cuh"

namespace specv {

constexpr int kC8Threads = 256 + 2 * 128;
constexpr uint32_t kC8TmemCols = 512;
constexpr int kC8Half = 128 * 128;  // 128 rows of one 64-column half: 16 KB
constexpr int kC8Issuer = 4;        // the warp among the first eight that issues the products
constexpr int kC8Loaders = 7;       // the others
// A row's sum over one tile up to which its reference stays, and where the reference is set below a maximum.
constexpr float kC8MaxSum = 65504.f;
constexpr float kC8HeadroomLog2 = 8.f;
// Units whose exponents are kept: the loaders are at most NS / 2 + 1 units ahead of the issuer, and the issuer
// one ahead of the softmax that it waits for.
constexpr int kC8Units = 16;
// How far the scales of a group's keys may lie apart for their values to be brought to the largest: e4m3's values are
// multiples of 2^-9, fp16's of 2^-24, so up to there nothing is lost.
constexpr int kC8Gap = 15;
// What scores are multiplied by at least: as sums below 2^31, they move by less than 2^-25.  Scores that the softmax has
// scaled by itself are put back divided by it, at most kC8Most of them.
constexpr float kC8LeastScale = 1.3877787807814457e-17f;  // 2^-56
constexpr float kC8Most = 1.1805916207174113e21f;         // 2^70

template <int D>
struct C8 {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kC8Half;       // a K or V tile, or a Q block
  // P has columns of its own where there are enough, so that S outlives it and the softmax can go over halves in a loop:
  // nothing spills (24 mixed sequences: 130 us without, 128.5 with)
  static constexpr bool kApart = D == 64;
  static constexpr int kStages = D == 128 ? 4 : 8;      // 128 KB; what is left is L1's
  static constexpr size_t kSmem = 1024 + 2 * (size_t)kTile + (size_t)kStages * kTile;
  static_assert(kSmem + 2048 <= 227 * 1024, "with the statically allocated part");
  static constexpr uint32_t kIdescQK = tc::idesc_f16(128, 128, 0, 0);
  static constexpr uint32_t kIdescPV = tc::idesc_f16(128, D, 0, 1);
};

__device__ __forceinline__ uint32_t c8_col_s(int w) { return 256u * w; }
__device__ __forceinline__ uint32_t c8_col_o(int w) { return 256u * w + 128u; }
template <int D>
__device__ __forceinline__ uint32_t c8_col_p(int w) { return C8<D>::kApart ? c8_col_o(w) + D : c8_col_s(w); }

// Units of the piece that block w's rows see: [b0, b1), empty for a block without rows.
__device__ __forceinline__ void c8_block_units(const ServeAttnParams& p, const PieceItem& it, int w, int& b0, int& b1) {
  const int rows = it.s.n * p.G, r0 = it.row0 + w * 128;
  b0 = b1 = it.u0;
  if (r0 >= rows) return;
  const int rl = min(r0 + 128, rows) - 1, base = it.s.len - it.s.n;
  const int first = p.window > 0 ? max(0, base + r0 / p.G + 1 - min(p.window, it.s.len)) : 0;
  b0 = max(it.u0, first / kTcKeys);
  b1 = max(b0, min(it.u1, (base + rl / p.G) / kTcKeys + 1));
}

template <int D, bool LIGHT>
__global__ void __launch_bounds__(kC8Threads, 1)
    chunk8_attn_tc(const __grid_constant__ Kv8Params p) {
  using C = C8<D>;
  constexpr int NS = C::kStages;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[NS], empty[NS];
  __shared__ uint64_t sfull[2], pfull[2], pvdone[2], ofree[2], qfull[2], drain;
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  // of a unit's four groups of 32 keys: K's scale, V's exponent, 1 / V's scale.  Where scales lie too far apart, V's
  // exponent is NaN and the last word says which (1 K's, 2 V's; 4: some of V's are far from 1) and their largest bytes
  __shared__ float4 s_scale[kC8Units][4], s_own[8][4];
  __shared__ LightSeqs s_light;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* qs = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // [block][half][128 rows][128 B]
  uint8_t* stages = qs + 2 * C::kTile;
  const uint32_t qs_u32 = smem_u32(qs), stages_u32 = smem_u32(stages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 4);  // the groups of a tile
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
  if (warp == kC8Issuer) tc::alloc(&tmem_base, kC8TmemCols);
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

  // registers: 256 x 96 + 256 x 160 = 512 x 128, what the block was launched with
  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp != kC8Issuer) {
    // ------------------------------------------------------------------ loaders
    // A group is 32 rows of a tile: 0-3 of a unit are K's, 4-7 V's, dealt to the warps in turn, so that a warp
    // has the time of seven groups for one group's loads.
    // lane: chunk lane & 3 (16 values) of a half of row i * 8 + lane / 4 of the group's 32.  Eight lanes then store
    // to eight different groups of banks: even chunks of an even row, odd ones of an odd row.
    constexpr int NH = C::kHalves;
    const int rl = lane >> 2, cl = lane & 3;
    // the group that is looked up
    int grp = warp < kC8Issuer ? warp : warp - 1, unit = 0, round = 0;
    int u = 0, u1 = 0, b = 0, g = 0, lo = 0, len = 0;
    auto open = [&]() {  // the next piece that has units; false at the end
      for (; round < rounds; ++round) {
        const PieceItem it = piece_item(list.fetch(p, round));
        if (it.u0 >= it.u1) continue;
        u = it.u0; u1 = it.u1; b = it.b; g = it.g; lo = it.s.lo; len = it.s.len;
        return true;
      }
      return false;
    };
    auto advance = [&]() {
      grp += kC8Loaders;
      if (grp < 8) return true;
      grp -= 8;
      ++unit;
      if (++u < u1) return true;
      ++round;
      return open();
    };
    // Nothing here looks at what it has just asked for: one wait for memory per group instead of three
    // (2048-token chunk at 32K: 812 us with them, 792 without).
    int page = 0, slot = 0;
    bool in = false;
    auto look_up = [&]() {  // page id and slot of this lane's key; it is looked at one group later
      const int t = u * kTcKeys + (grp & 3) * 32 + lane;
      in = t >= lo && t < len;
      if (!in) return;
      const int col = page_of(p, t);
      slot = t - col * p.page_size;
      page = __ldg(p.table + (int64_t)b * p.table_stride + col);
    };
    // the group that comes next: where its rows lie, and its exponents on their way
    int64_t off[4];
    const uint8_t* base = nullptr;
    int coming = 0;                   // unit * 8 + group
    bool live = false;                // this lane's key has a page
    uint32_t byte = 0, v_byte = 0;    // its exponent; a K group also looks after V's
    // Rows of 64: its addresses are made before the present group is stored, and its loads go out right behind (24 mixed
    // sequences 133.3 us without, 130.5 with).  Rows of 128 do not wait for memory most (a 2048-token chunk at 32K 789 and 796 us).
    constexpr bool kEarly = D == 64;
    uint4 raw[4 * NH];
    auto load = [&](int i) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
        raw[i * NH + h] = off[i] >= 0 ? __ldcg(reinterpret_cast<const uint4*>(base + off[i] + h * 64)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto load_all = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) load(i);
    };
    auto prepare = [&]() {
      coming = unit * 8 + grp;
      live = in && page >= 0 && page < p.num_pages;
      if (in && !live) chunk_report<LIGHT>(p, (uint32_t)SPEC_STATUS_BAD_PAGE);
      __syncwarp();
      const int64_t mine = live ? (int64_t)page * p.kv_sp + (int64_t)slot * p.kv_st + (int64_t)g * p.kv_sh : -1;
      base = reinterpret_cast<const uint8_t*>(grp < 4 ? p.k : p.v) + cl * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        off[i] = __shfl_sync(0xffffffffu, mine, i * 8 + rl);
        if constexpr (!kEarly) load(i);
      }
      if (live) {
        const int64_t at = (int64_t)page * p.exp_sp + (int64_t)g * p.exp_sh + block_of(p, slot);
        byte = (grp < 4 ? p.k_exp : p.v_exp)[at];
        if (grp < 4) v_byte = p.v_exp[at];
      }
    };
    bool have = open();  // a group is looked up
    if (have) look_up();
    auto next = [&]() {
      if (!have) return false;
      prepare();
      have = advance();
      if (have) look_up();
      return true;
    };
    bool more = next();
    if (kEarly && more) load_all();
    while (more) {
      const int now = coming, mine = live ? clamp_exp((int)byte) : 0;
      const int top = __reduce_max_sync(0xffffffffu, mine);
      const bool apart = __any_sync(0xffffffffu, live && mine + kC8Gap < top);
      const bool uneven = __any_sync(0xffffffffu, live && mine != top) && !apart;
      const int step = now >> 2, s = step % NS;
      if ((now & 7) < 4) {
        // both exponents go out with K, before the scores that need them exist
        const int v_mine = live ? clamp_exp((int)v_byte) : 0;
        const int vtop = __reduce_max_sync(0xffffffffu, v_mine);
        const bool v_own = __any_sync(0xffffffffu, live && v_mine < max(vtop - kC8Gap, kFarLow)) || vtop > kFarHigh;
        const bool v_apart = v_own && __any_sync(0xffffffffu, live && v_mine + kC8Gap < vtop);
        if (lane == 0) {
          const int ke = top ? top - 127 : 0, ve = vtop ? vtop - 127 : 0, own = (int)apart | (int)v_apart << 1 | (int)v_own << 2;
          s_scale[(now >> 3) % kC8Units][now & 3] =
              make_float4(exp2_whole(ke), own ? __int_as_float(0x7fffffff) : (float)ve, exp2_whole(-ve),
                          __int_as_float(own ? own | top << 8 | vtop << 16 : 0));
        }
      }
      if constexpr (kEarly) more = next();
      const bool got = mbar_wait_spin(&empty[s], ((step / NS) & 1) ^ 1u, &s_abort);
      if (!__all_sync(0xffffffffu, got)) {
        fail();
        break;
      }
      const uint32_t dst = stages_u32 + s * C::kTile + ((now & 3) * 32 + rl) * 128;
      // two straight pieces of code: with the choice inside, each chunk's stores wait for its conversions
      auto rows = [&](auto scaled) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __half2 f;
          if constexpr (scaled.value) f = __float2half2_rn(exp2_whole(max(__shfl_sync(0xffffffffu, mine, i * 8 + rl) - top, -kC8Gap)));
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const uint32_t w[4] = {raw[i * NH + h].x, raw[i * NH + h].y, raw[i * NH + h].z, raw[i * NH + h].w};
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16x4(w[e], v[2 * e], v[2 * e + 1]);
            if constexpr (scaled.value) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&v[e]), f);
                v[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
            const uint32_t row = dst + h * kC8Half + i * 1024;  // (row & 7) == rl
            sts128(row + (((2 * cl) ^ rl) << 4), v[0], v[1], v[2], v[3]);
            sts128(row + (((2 * cl + 1) ^ rl) << 4), v[4], v[5], v[6], v[7]);
          }
        }
      };
      if (uneven) rows(std::true_type{});
      else rows(std::false_type{});
      tc::fence_proxy_async_smem();  // every lane's stores, for the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      if constexpr (!kEarly) more = next();
      else if (more) load_all();
    }
    } else {
    // ------------------------------------------------------------------ MMA issuer (one lane)
    if (elect_one()) {
      int step = 0, part[2] = {0, 0}, t[2] = {0, 0};  // pieces and tiles so far, by block
      bool ok = true;
      // S_w = Q_w K^T (behind P_w V of the tile before, whose P it overwrites)
      const uint32_t q_lo = tc::desc_lo(qs_u32, 16), k_lo = tc::desc_lo(stages_u32, 16);
      const uint32_t v_lo = tc::desc_lo(stages_u32, kC8Half);
      auto issue_qk = [&](int w, int stage) {
        const uint32_t qa = q_lo + w * (C::kTile >> 4), kb = k_lo + stage * (C::kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t koff = ((ks >> 2) * kC8Half + (ks & 3) * 32) >> 4;
          tc::mma_ss_lo(tmem + c8_col_s(w), qa + koff, kb + koff, C::kIdescQK, ks > 0 ? 1u : 0u);
        }
        tc::commit(&sfull[w]);
      };
      PieceRaw ahead = list.fetch(p, 0);
      for (int round = 0; ok && round < rounds; ++round) {
        const PieceItem it = piece_item(ahead);
        ahead = list.fetch(p, round + 1);
        if (it.u0 >= it.u1) continue;
        int b0[2], b1[2];
        c8_block_units(p, it, 0, b0[0], b1[0]);
        c8_block_units(p, it, 1, b0[1], b1[1]);
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
                tc::mma_ts_lo(tmem + c8_col_o(w), tmem + c8_col_p<D>(w) + ks * 8, vb + ks * (2048 >> 4), C::kIdescPV,
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
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    // ------------------------------------------------------------------ softmax warpgroups
    const int w = (warp - 8) >> 2;
    const int sub = warp & 3;        // TMEM sub-partition of this warp
    const int m = sub * 32 + lane;   // TMEM lane = row of the block
    const uint32_t tl = tmem + ((uint32_t)(sub * 32) << 16);
    const uint32_t sbuf = tl + c8_col_s(w), pbuf = tl + c8_col_p<D>(w), obuf = tl + c8_col_o(w);
    const uint32_t qblock_u32 = qs_u32 + w * C::kTile;
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool got = mbar_wait_spin(bar, parity, &s_abort);
      return __all_sync(0xffffffffu, got);
    };
    // the next piece in which this block has tiles; pieces without leave an empty record.  `units`: units of the
    // list before piece `round`, `nbase`: before the piece returned
    int round = 0, units = 0, nbase = 0;
    PieceRaw ahead = list.fetch(p, 0);
    auto next_piece = [&](PieceItem& n, int& nb0, int& nb1) -> bool {
      while (round < rounds) {
        n = piece_item(ahead);
        ahead = list.fetch(p, ++round);
        nbase = units - n.u0;
        units += max(n.u1 - n.u0, 0);
        c8_block_units(p, n, w, nb0, nb1);
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
        cp_async16(qblock_u32 + (c >> 3) * kC8Half + (sub * 32 + row) * 128 + (((c & 7) ^ (row & 7)) << 4),
                   reinterpret_cast<const __nv_bfloat16*>(p.q) + (off < 0 ? 0 : off) + c * 8, off >= 0);
      }
      cp_async_commit();
    };
    // the rows, once they have landed, to fp16 in place, each scaled by a power of two; returns what the scores of
    // this thread's row are multiplied by
    auto finish_q = [&]() -> float {
      constexpr int CH = D / 8, RPI = 32 / CH;
      cp_async_wait<0>();
      const int c = lane % CH;
      float mine = 0.f;
#pragma unroll 2
      for (int i = 0; i < 32 / RPI; ++i) {
        const int row = i * RPI + lane / CH;
        const uint32_t at = qblock_u32 + (c >> 3) * kC8Half + (sub * 32 + row) * 128 + (((c & 7) ^ (row & 7)) << 4);
        uint32_t v[4];
        lds128(at, v[0], v[1], v[2], v[3]);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmax3(amax, fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u)));
#pragma unroll
        for (int x = 1; x < CH; x <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
        float undo;
        const float up = f16_scale(amax, undo);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = pack_f16(__uint_as_float(v[e] << 16) * up, __uint_as_float(v[e] & 0xffff0000u) * up);
        sts128(at, v[0], v[1], v[2], v[3]);
        undo = __shfl_sync(0xffffffffu, undo, lane % RPI * CH);
        if (lane / RPI == i) mine = q_factor(undo, p.scale_log2);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[w]);
      return mine;
    };

    PieceItem it;
    int b0 = 0, b1 = 0, tok = -1, head = 0;
    bool have = next_piece(it, b0, b1), ok = true;
    int base = nbase, cur = round - 1;  // the piece's place in the list
    float qscale = 0.f;
    if (have) {
      start_q(it, tok, head);
      qscale = finish_q();
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
        // what the scores of 32 columns are multiplied by; hidden scores stay -inf
        const float4* scales = s_scale[(base + u) % kC8Units];
        auto k_scale = [&](const float4& x) { return fmaxf(qscale * x.x, kC8LeastScale); };
        // The usual tile is straight code of a few hundred instructions, 32 columns at a time with the next ones on
        // their way (with all 128 in registers beside P the kernel spills, and what spills goes to L2, because
        // shared memory leaves L1 nothing).  What is rare goes over S in TMEM before it, in loops: hidden
        // scores become -inf there, and the maximum is taken there.
        if (edge) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int h = hi - c * 32, l = lo - c * 32;  // visible [l, h]
            const uint32_t vis = (h >= 31 ? ~0u : h < 0 ? 0u : (2u << h) - 1u) & (l <= 0 ? ~0u : l > 31 ? 0u : ~0u << l);
            if (__all_sync(0xffffffffu, vis == ~0u)) continue;
            uint32_t v[32];
            tc::ld32(sbuf + c * 32, v);
            tc::ld_wait(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (vis >> e) & 1u ? v[e] : 0xff800000u;
            tc::st32(sbuf + c * 32, v);
          }
          tc::st_wait();
        }
        // P = 2^(s + ev - mu) against the present reference, as fp16 pairs; only where a row's sum says that a
        // score lies far above it (or nothing has been seen yet) is the tile's maximum taken, O rescaled and
        // the tile done again.  Keys with scales of their own make the sum a NaN, which comes that way, too: S then
        // becomes what their scores are, and they are counted apart
        uint32_t pk[C::kApart ? 32 : 64];
        float sum, lsum;
        bool exact = u == b0;
        for (;;) {
          if (exact) {
            float top = neg_inf();
            uint32_t own = 0u;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              tc::ld32(sbuf + c * 32, v);
              tc::ld_wait(v);
              float mx = neg_inf();
#pragma unroll
              for (int e = 0; e < 32; e += 2) mx = fmax3(mx, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              const float4 x = scales[c];
              if (mx != neg_inf()) top = fmaxf(top, fmaf(mx, k_scale(x), x.y));  // not where x.y is NaN
              own |= __float_as_uint(x.w);
            }
            float own_top = -kC8Most, own_sum = 0.f;  // a bound on s, and the sum of 2^(s - it)
            if (own) {
              const PieceItem at = piece_item(list.fetch(p, cur));
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const uint32_t w = __float_as_uint(scales[c].w);
                if (!w) continue;
                // the lane's key's bytes, K's below V's, looked up once more (a place for all in shared memory would
                // leave L1 a step less of it: 830 us instead of 799 for a 2048-token chunk at 32K)
                uint32_t mine = 0u;
                const int t = u * kTcKeys + c * 32 + lane;
                if (t >= at.s.lo && t < at.s.len) {
                  int page, slot;
                  page_slot(p, at.b, t, page, slot);
                  if (page >= 0) {
                    const int64_t place = (int64_t)page * p.exp_sp + (int64_t)at.g * p.exp_sh + block_of(p, slot);
                    mine = (uint32_t)clamp_exp(p.k_exp[place]) | (uint32_t)clamp_exp(p.v_exp[place]) << 8;
                  }
                }
                if (!(w & 1u)) mine = (mine & 0xff00u) | (w >> 8 & 0xffu);
                if (!(w & 2u)) mine = (mine & 0xffu) | (w >> 8 & 0xff00u);
#pragma unroll 1
                for (int d = 0; d < 32; d += 8) {
                  uint32_t v[8];
                  tc::ld8_wait(sbuf + c * 32 + d, v);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const uint32_t b = __shfl_sync(0xffffffffu, mine, d + e);
                    const float s = __uint_as_float(v[e]) * fmaxf(qscale * __uint_as_float((b & 0xffu) << 23), 1.17549435e-38f);
                    const float z = s + (float)((int)(b >> 8) - 127), to = fmaxf(own_top, s);
                    top = fmaxf(top, z);
                    own_sum = own_sum * ex2_approx(own_top - to) + ex2_approx(s - to);
                    own_top = to;
                    if (s != neg_inf()) v[e] = __float_as_uint(fminf(fmaxf(z, -kC8Most), kC8Most) * (1.f / kC8LeastScale));
                  }
                  tc::st8(sbuf + c * 32 + d, v);
                }
              }
              tc::st_wait();
              if (lane < 4) s_own[warp - 8][lane] = scales[lane].w != 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : scales[lane];
              __syncwarp();
              scales = s_own[warp - 8];
            }
            const float m_new = top == neg_inf() ? m_run : fmaxf(m_run, top - kC8HeadroomLog2);
            const float alpha = m_run == neg_inf() ? 0.f : ex2_approx(m_run - m_new);
            l = m_run == neg_inf() ? 0.f : scale_sum(l, m_run - m_new, alpha);
            if (own_sum > 0.f) l = fmaf(own_sum, ex2_approx(own_top - m_new), l);
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
          const float mu = m_run == neg_inf() ? 0.f : m_run;
          sum = lsum = 0.f;
          auto chunk = [&](const uint32_t(&v)[32], int c, int at) {  // columns 32 c .. to pk[at ..]
            const float4 x = scales[c];
            const float scale = k_scale(x), nmu = x.y - mu;
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              fma2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), scale, nmu, x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              add2(sums[e & 2], sums[(e & 2) + 1], p0, p1);
              pk[at + e / 2] = pack_f16(p0, p1);
            }
            const float part = (sums[0] + sums[1]) + (sums[2] + sums[3]);
            sum += part;
            lsum = fmaf(part, x.z, lsum);
          };
          uint32_t sa[32], sb[32];
          if constexpr (C::kApart) {
#pragma unroll 1
            for (int c = 0; c < 4; c += 2) {
              tc::ld32(sbuf + c * 32, sa);
              tc::ld_wait(sa);
              tc::ld32(sbuf + c * 32 + 32, sb);
              chunk(sa, c, 0);
              tc::ld_wait(sb);
              chunk(sb, c + 1, 16);
              tc::st32(pbuf + c * 16, reinterpret_cast<uint32_t(&)[32]>(pk[0]));
            }
          } else {
            tc::ld32(sbuf, sa);
            tc::ld_wait(sa);
            tc::ld32(sbuf + 32, sb);
            chunk(sa, 0, 0);
            tc::ld_wait(sb);
            tc::ld32(sbuf + 64, sa);
            chunk(sb, 1, 16);
            tc::ld_wait(sa);
            tc::ld32(sbuf + 96, sb);
            chunk(sa, 2, 32);
            tc::ld_wait(sb);
            chunk(sb, 3, 48);
          }
          if (exact || !__any_sync(0xffffffffu, !(sum <= kC8MaxSum) || m_run == neg_inf())) break;
          exact = true;
        }
        l += lsum;
        __syncwarp();
        if constexpr (!C::kApart) {
          tc::st32(pbuf, reinterpret_cast<uint32_t(&)[32]>(pk[0]));
          tc::st32(pbuf + 32, reinterpret_cast<uint32_t(&)[32]>(pk[32]));
        }
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
      float next_scale = 0.f;
      if (have_next) next_scale = finish_q();
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
        const int up = sum_shift(l);
        const float f = exp2_whole(-up);
        float* dst = p.part_o + rec * D * kTcRows + w * 128 + m;
        uint32_t v[32];
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          __syncwarp();
          tc::ld32(obuf + c * 32, v);
          tc::ld_wait(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) dst[(c * 32 + e) * kTcRows] = __uint_as_float(v[e]) * f;
        }
        p.part_ml[rec * kTcRows + w * 128 + m] = make_float2(m_run + up, l * f);
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
      base = nbase;
      cur = round - 1;
      qscale = next_scale;
      b0 = nb0;
      b1 = nb1;
      tok = ntok;
      head = nhead;
    }
    if (!ok) fail();
  }

  tc::fence_before();
  __syncthreads();
  if (warp == kC8Issuer) {
    __syncwarp();
    tc::fence_after();
    tc::dealloc(tmem, kC8TmemCols);
  }
}

template <int D, bool LIGHT>
static cudaError_t launch_tc8(const Kv8Params& p, cudaStream_t stream) {
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(chunk8_attn_tc<D, LIGHT>), (int)C8<D>::kSmem);
  if (e != cudaSuccess) return e;
  if (p.first) {
    chunk8_attn_tc<D, LIGHT><<<p.grid, kC8Threads, C8<D>::kSmem, stream>>>(p);
    return cudaGetLastError();
  }
  return launch_dependent(chunk8_attn_tc<D, LIGHT>, dim3(p.grid), dim3(kC8Threads), C8<D>::kSmem, stream, 0u, p);
}

cudaError_t launch_chunk8_tc(const Kv8Params& p, cudaStream_t stream) {
  if (p.light) return p.D == 128 ? launch_tc8<128, true>(p, stream) : launch_tc8<64, true>(p, stream);
  return p.D == 128 ? launch_tc8<128, false>(p, stream) : launch_tc8<64, false>(p, stream);
}

}  // namespace specv
