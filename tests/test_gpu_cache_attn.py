"""GPU parity of spec_paged_attn8 against the float64 oracle, element by element.

Tolerance of an output element, derived.  With A = sum_t p_t |v_t| and r the largest relative error of a probability
before its rounding, the numerator's and the normaliser's shares are at most 2 r A.  r: the score is a D-term
fp32 sum, off by at most (D + 8) 2^-24 S with S the largest scale * sum |q k| (absolutely: it sits in an exponent), the
exponents up to 64 of V's scales are added to it in fp32 (2^-23 * 64, twice), and 2^-20 for 2^x and the
running rescales.  Probabilities are rounded to fp16: 2^-11 A, and where they are below 2^-14 by half a step of 2^-24;
as the largest p' = c p 2^ev is at least 2^7, that moves the output by at most sum 2^-25 |v / 2^ev| / c <= 2^-32 W, with
W = max(p 2^ev) * sum |v / 2^ev|.  In large chunks 32 neighbouring keys have one ev, the largest of theirs, and the
values v / 2^ev that go with it; W holds both forms.  The P.V and l sums over L keys add L 2^-24 A each; the output's
own rounding comes last.  Values brought to a neighbour's scale up to 2^14 above their own lose nothing in fp16
(e4m3's are multiples of 2^-9, fp16's of 2^-24).  Slots past kv_len and pages before the window hold NaN codes."""

import numpy as np
import pytest

from oracle import cache as oc

from .helpers import torch_mod
from .test_gpu_cache import SENTINEL, Cache8, dt, i32, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def check(o, ref, A, W, S, D, L, o_dtype, what=""):
    r = (D + 8) * 2.0 ** -24 * S + 2.0 ** -16 + 2.0 ** -20
    tol = (2 * r + 2 * L * 2.0 ** -24 + 2.0 ** -11) * A + 2.0 ** -32 * W
    tol = tol + (2.0 ** -8 if o_dtype == "bf16" else 2.0 ** -24) * np.abs(ref) + 1e-30
    assert np.all(np.isfinite(o)), f"{what}: non-finite output"
    over = np.abs(o - ref) / tol
    assert over.max(initial=0) <= 1, f"{what}: {over.max():.3g} times the bound at {np.unravel_index(over.argmax(), over.shape)}"


class Attn(Cache8):
    """A cache whose unseen slots are NaN, queries, and optionally new rows to append."""

    def __init__(self, q_len, kv_len, G=4, window=0, append=False, exp_lo=117, exp_hi=121, q_scale=1.0, **kw):
        torch = torch_mod()
        super().__init__(q_len, kv_len, **kw)
        self.window, self.do_append, self.G = window, append, G
        rng = self.rng
        seen = np.zeros((self.pages, self.page), bool)
        for b in range(self.B):
            n, length = int(q_len[b]), int(kv_len[b])
            lo = max(0, length - n + 1 - window) if window else 0
            if n == 0:
                continue
            for t in range(lo, length - n if append else length):
                seen[self.table[b, t // self.page], t % self.page] = True
            if window:
                self.table[b, :lo // self.page] = -5  # given back
        small = np.array([c for c in range(256) if c & 127 <= 0x70], dtype=np.uint8)
        for c, e in zip(self.codes, self.exps):
            c[:] = np.where(seen[:, None, :, None], small[rng.integers(0, len(small), c.shape)], 0x7F)
            e[:] = rng.integers(exp_lo, exp_hi + 1, e.shape)
        self.q = torch.from_numpy(rng.standard_normal((self.T, G * self.Hkv, self.D)) * q_scale).bfloat16()
        self.q[:self.start[0]] = float("nan")
        self.q[self.start[-1]:] = float("nan")
        self.max_q = max(max(q_len), 1)

    def reference(self):
        codes, exps = self.codes, self.exps
        if self.do_append:
            *both, = oc.append8(*(np64(x) for x in self.new), *codes, *exps, self.table, self.start, self.kv_len, self.block)
            codes, exps = both[:2], both[2:]
        return oc.paged_attn8(np64(self.q), codes, exps, self.table, self.start, self.kv_len, self.window), (*codes, *exps)

    def run(self, sv, o_dtype="f32", o=None, max_q=None, **kw):
        torch = torch_mod()
        self.to_device()
        self.d_q = self.q.cuda()
        if o is None:
            o = torch.full(self.q.shape, SENTINEL, dtype=dt(o_dtype), device="cuda")
        max_q = max_q or self.max_q
        need = sv.spec_paged_attn8_workspace(self.d_q, self.d_codes[0], self.d_table, o, max_q=max_q)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        new = dict(k_new=self.d_new[0], v_new=self.d_new[1]) if self.do_append else {}
        sv.spec_paged_attn8(self.d_q, *self.d_codes, *self.d_exps, self.d_table, self.d_start, self.d_len, o, max_q=max_q,
                            window=self.window, workspace=ws, **new, **kw)
        torch.cuda.synchronize()
        return np64(o), sv.read_status(ws)

    def verify(self, sv, o_dtype="f32", what="", **kw):
        (ref, A, W, S), state = self.reference()
        o, st = self.run(sv, o_dtype, **kw)
        r0, r1 = self.start[0], self.start[-1]
        assert st == 0
        check(o[r0:r1], ref[r0:r1], A[r0:r1], W[r0:r1], S, self.D, int(self.kv_len.max()), o_dtype, what)
        assert np.all(o[:r0] == SENTINEL) and np.all(o[r1:] == SENTINEL)
        for got, want in zip(self.state(), state):
            assert np.array_equal(got, want)
        return o


SMALL = [
    dict(q_len=[1], kv_len=[1], G=1), dict(q_len=[1], kv_len=[300], D=128), dict(q_len=[1, 1, 1], kv_len=[15, 16, 17], page=16),
    dict(q_len=[5, 0, 3, 1], kv_len=[700, 40, 3, 129], D=128), dict(q_len=[8, 2], kv_len=[1000, 2], page=24, block=12),
    dict(q_len=[4] * 3, kv_len=[4, 200, 513], G=8, D=128, page=128, block=1), dict(q_len=[3, 9], kv_len=[77, 600], G=3, page=7, block=7),
    dict(q_len=[1] * 70, kv_len=[20 + 13 * i for i in range(70)], Hkv=1), dict(q_len=[1], kv_len=[9000], G=32, Hkv=1),
    dict(q_len=[2, 2], kv_len=[3000, 2500], page=64, block=32, layout="nhd", D=128, Hkv=3)]
LARGE = [
    dict(q_len=[33], kv_len=[33], G=1), dict(q_len=[40, 0, 1, 9], kv_len=[700, 90, 130, 9], D=128),
    dict(q_len=[70, 100], kv_len=[300, 100], page=24, block=12), dict(q_len=[64], kv_len=[1500], G=8, D=128, Hkv=1, page=128, block=128),
    dict(q_len=[129, 5], kv_len=[129, 400], G=3, page=64, block=1, Hkv=1), dict(q_len=[300], kv_len=[2000], G=2, page=7, block=7, Hkv=1),
    dict(q_len=[20] * 70, kv_len=[20 + 5 * i for i in range(70)], Hkv=1, G=2), dict(q_len=[16, 90], kv_len=[2100, 1200], D=128, G=4, layout="nhd", page=32, block=4),
    dict(q_len=[35, 34], kv_len=[4000, 35], G=1, Hkv=5, page=16, block=16)]


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("kw", SMALL + LARGE)
def test_attention_parity(sv, kw, window, append):
    Attn(**kw, window=window, append=append, seed=len(kw["q_len"]) + kw["kv_len"][0]).verify(sv, "bf16" if window else "f32")


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 24, 25, 32, 33, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_at_tile_boundaries(sv, rows, D):
    Attn([rows, 1], [rows + 140, 70], G=1, Hkv=2, D=D, seed=rows).verify(sv)


@pytest.mark.parametrize("length", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 511, 512, 513, 640])
@pytest.mark.parametrize("q", [1, 40])
def test_lengths_at_tile_boundaries(sv, length, q):
    n = min(q, length)
    Attn([n], [length], G=4 if q == 1 else 1, Hkv=2, D=128, page=16, block=16, seed=length).verify(sv, max_q=q)


@pytest.mark.parametrize("q_len", [[3], [60]])
def test_scales_far_apart(sv, q_len):
    """V scales from 2^-60 to 2^60 from block to block: the outputs follow the largest that a row weighs."""
    c = Attn(q_len, [400], G=4, Hkv=2, D=64, page=32, block=32, seed=3)
    c.exps[1][:] = c.rng.integers(67, 188, c.exps[1].shape)
    c.verify(sv)


def test_scale_bytes_beyond_the_range(sv):
    """Bytes outside [63, 191] count as the nearest of them."""
    for q_len in ([2], [50]):
        c = Attn(q_len, [200], G=4, Hkv=1, D=64, page=32, block=32, seed=3)
        c.exps[0][:] = c.rng.choice([0, 30, 63], c.exps[0].shape)
        c.exps[1][:] = c.rng.choice([191, 192, 255], c.exps[1].shape)
        c.verify(sv)


@pytest.mark.parametrize("q_len", [[4], [70]])
def test_uneven_scales_among_32_keys(sv, q_len):
    """Blocks of one token whose scales lie up to 2^20 apart: in tiles of the tensor core the small ones are brought to
    their neighbours' scale in fp16, where a value is off by at most 2^-25 of it."""
    c = Attn(q_len, [300], G=4, Hkv=1, D=64, page=32, block=1, seed=6, q_scale=0.05)
    for e in c.exps:
        e[:] = c.rng.integers(100, 121, e.shape)
    (ref, A, W, S), _ = c.reference()
    o, st = c.run(sv)
    r0, r1 = c.start[0], c.start[-1]
    # scores: 2^-25 2^ktop sum |q|; values: 2^-25 2^vtop, over all keys at most
    q1 = np.abs(np.nan_to_num(np64(c.q))).sum(-1).max() * 64 ** -0.5
    extra = 2 * 2.0 ** -25 * 2.0 ** -7 * q1 * A + 2.0 ** -25 * 2.0 ** -7
    assert st == 0 and 2 * 2.0 ** -25 * q1 < 1e-6
    D, L = 64, 300
    tol = (2 * ((D + 8) * 2.0 ** -24 * S + 2.0 ** -16 + 2.0 ** -20) + 2 * L * 2.0 ** -24 + 2.0 ** -11) * A + 2.0 ** -32 * W + extra + 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(o - ref)[r0:r1] <= tol[r0:r1])


@pytest.mark.parametrize("q_scale", [2.0 ** -60, 2.0 ** 30])
@pytest.mark.parametrize("q_len", [[3], [60]])
def test_query_magnitudes(sv, q_len, q_scale):
    """Rows far outside fp16's range: scores stay as they are because the scale goes the other way."""
    c = Attn(q_len, [200], G=4, Hkv=2, D=64, seed=4)
    base = c.reference()[0]
    c.q = (c.q.float() * q_scale).bfloat16()
    o, st = c.run(sv, scale=64 ** -0.5 / q_scale)
    r0, r1 = c.start[0], c.start[-1]
    check(o[r0:r1], base[0][r0:r1], base[1][r0:r1], base[2][r0:r1], base[3], 64, 200, "f32")


def test_sharp_and_rising_scores(sv):
    """Scores that rise by hundreds along the keys, so that the reference has to move again and again."""
    for q_len in ([2], [64]):
        c = Attn(q_len, [700], G=4, Hkv=1, D=64, page=64, block=64, seed=5, q_scale=0.0)
        c.q[c.start[0]:c.start[-1], :, 0] = 1.0
        for t in range(700):
            page, slot = c.table[0, t // 64], t % 64
            c.codes[0][page, :, slot] = 0
            c.codes[0][page, :, slot, 0] = oc.encode(float(t % 449))
            c.exps[0][page] = 127
        c.verify(sv)
        c.codes[0][:, :, :, 0] = 0
        c.verify(sv)  # all scores alike


def test_padding_bound_of_max_q(sv):
    """max_q above every chunk: the kernels for more rows take calls of few."""
    c = Attn([1, 5], [100, 333], D=128, seed=8)
    c.verify(sv)
    c.verify(sv, max_q=500)


@pytest.mark.parametrize("big", [1, 60])
def test_bad_data(sv, big):
    c = Attn([big, big, big, big], [300, big - 1 if big > 1 else 0, 200, 250], seed=3)
    c.kv_len[3] = c.table.shape[1] * c.page + 1
    c.table[2, 3] = c.pages + 1
    o, st = c.run(sv)
    s = c.start
    assert st == sv.SPEC_STATUS_BAD_KV_LEN | sv.SPEC_STATUS_BAD_PAGE
    assert np.all(o[s[1]:s[2]] == 0) and np.all(o[s[3]:s[4]] == 0)
    own = Attn([big, big, big, big], [300, big - 1 if big > 1 else 0, 200, 250], seed=3)
    (ref, A, W, S) = oc.paged_attn8(np64(own.q), own.codes, own.exps, own.table, own.start[:2], own.kv_len[:1])
    check(o[s[0]:s[1]], ref[s[0]:s[1]], A[s[0]:s[1]], W[s[0]:s[1]], S, 64, 300, "f32")
    c = Attn([big, big, big], [100, 100, 100], seed=4)
    c.start[1] = c.start[2] + 1
    o, st = c.run(sv)
    assert st & sv.SPEC_STATUS_BAD_RANGE


@pytest.mark.parametrize("q_len", [[5, 1, 3], [50, 0, 37]])
def test_strided_output_and_queries(sv, q_len):
    torch = torch_mod()
    c = Attn(q_len, [300, 90, 200], Hkv=2, G=4, seed=12)
    want = c.verify(sv)
    T = c.T
    wide = torch.full((8, T, 64 + 3), SENTINEL, dtype=torch.float32, device="cuda")
    o = wide[:, :, 1:65].transpose(0, 1)
    got, _ = c.run(sv, o=o)
    assert np.array_equal(got[c.start[0]:c.start[-1]], want[c.start[0]:c.start[-1]])
    assert bool((wide[:, :, 0] == SENTINEL).all()) and bool((wide[:, :, 65:] == SENTINEL).all())
    fused = torch.zeros(T, 12, 64, dtype=torch.bfloat16)
    fused[:, :8] = c.q
    c.q = fused[:, :8]
    got, _ = c.run(sv)
    assert np.array_equal(got[c.start[0]:c.start[-1]], want[c.start[0]:c.start[-1]])


@pytest.mark.parametrize("q_len,kv_len", [([5, 1], [900, 333]), ([1], [200]), ([60, 9], [500, 700]), ([40], [90])])
def test_repeats_streams_and_graphs(sv, q_len, kv_len):
    """The same bits every time: again, on another stream, from a graph whose inputs changed in between."""
    torch = torch_mod()
    c = Attn(q_len, kv_len, append=True, D=128, seed=13)
    want, _ = c.run(sv)
    after = c.state()
    again, _ = c.run(sv)
    assert np.array_equal(want, again)
    c.to_device()
    o = torch.empty(c.q.shape, dtype=torch.float32, device="cuda").fill_(SENTINEL)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda out, **kw: sv.spec_paged_attn8(c.d_q, *c.d_codes, *c.d_exps, c.d_table, c.d_start, c.d_len, out,  # noqa: E731
                                                 max_q=c.max_q, k_new=c.d_new[0], v_new=c.d_new[1], **kw)
    call(o, stream=side)
    side.synchronize()
    assert np.array_equal(np64(o), want)
    for x, y in zip(c.state(), after):
        assert np.array_equal(x, y)
    c.to_device()
    g = torch.cuda.CUDAGraph()
    o2 = torch.empty_like(o).fill_(SENTINEL)
    with torch.cuda.graph(g, stream=side):
        call(o2)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(np64(o2), want)
    c.d_q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    c.q = c.d_q.cpu()
    c.codes, c.exps = after[:2], after[2:]
    o3, _ = c.run(sv)
    assert np.array_equal(np64(o2), o3)


def test_a_serving_step_end_to_end(sv):
    """Beams forked, positions turned, K/V appended and attended to, pages compacted, step after step, against the
    oracles of each; prompts are cached by spec_kv8_append after spec_prefill_attn."""
    torch = torch_mod()
    rng = np.random.default_rng(20)
    B, Hq, Hkv, D, page, block, pages, cols = 4, 4, 2, 64, 16, 8, 64, 12
    e4 = lambda: torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    kp, vp = e4(), e4()
    ke, ve = (torch.full((pages, Hkv, page // block), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    raw = lambda: [x.view(torch.uint8).cpu().numpy().copy() for x in (kp, vp, ke, ve)]  # noqa: E731
    table, held, lens, refs = i32(np.zeros((B, cols))), i32([0] * B), i32([0] * B), i32([0] * pages)
    steps, _ = sv.spec_rotary_steps(D)
    f = steps.cpu().numpy().astype(np.longdouble) / np.longdouble(2.0) ** 64 * 2 * np.longdouble(np.pi)
    fork = lambda parent, grow: sv.spec_page_fork(table, held, lens, refs, i32(parent), page_size=page, grow=i32(grow),  # noqa: E731
                                                  caches=[kp, vp, ke, ve])
    host = [x.cpu().numpy() for x in (table, held, lens, refs)]
    for step, (parent, grow) in enumerate([([0, 1, -1, -1], [40, 21, 0, 0]), ([0, 0, 1, 0], [1, 1, 1, 1]), ([2, 1, 2, 3], [5, 0, 3, 1]),
                                           ([0, 1, -1, 3], [1, 1, 0, 1]), ([0, 3, 3, 3], [35, 2, 2, 2])]):
        before = raw()
        fork(parent, grow)
        want = oc.page_fork(*host, parent, grow, page)
        host = list(want[:4])
        for x in before:
            for a, b in want[4]:
                x[b] = x[a]
        for x, y in zip((table, held, lens, refs), host):
            assert np.array_equal(x.cpu().numpy(), y)
        assert all(np.array_equal(x, y) for x, y in zip(raw(), before))
        grow = [g if p >= 0 else 0 for p, g in zip(parent, grow)]
        T = sum(grow)
        start = np.cumsum([0] + grow)
        q, k, v = (torch.from_numpy(rng.standard_normal((T, H, D))).bfloat16().cuda() for H in (Hq, Hkv, Hkv))
        q0, k0 = np64(q), np64(k)
        sv.spec_rotary(q, k, steps, q_start=i32(start), kv_len=lens)
        pos = np.concatenate([np.arange(n - g, n) for n, g in zip(host[2], grow)])
        for x, x0 in ((q, q0), (k, k0)):
            ref = oc.rotary(x0, pos, f, False)
            assert np.abs(np64(x) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -18 * np.abs(x0).max()
        o = torch.empty_like(q, dtype=torch.float32)
        new = (np64(k), np64(v))
        state = oc.append8(*new, *before, host[0], start, host[2], block)
        if step == 0:  # prompts: attention over the rows themselves, then the cache
            sv.spec_prefill_attn(q, k, v, i32(start), o)
            sv.spec_kv8_append(k, v, kp, vp, ke, ve, table, i32(start), lens)
        else:
            sv.spec_paged_attn8(q, kp, vp, ke, ve, table, i32(start), lens, o, max_q=max(grow), k_new=k, v_new=v)
            ref, A, W, S = oc.paged_attn8(np64(q), state[:2], state[2:], host[0], start, host[2])
            check(np64(o), ref, A, W, S, D, int(host[2].max()), "f32", f"step {step}")
        assert all(np.array_equal(x, y) for x, y in zip(raw(), state))
        if step == 3:
            sv.spec_page_compact(table, held, refs, caches=[kp, vp, ke, ve])
            t, r, _, live, copies = oc.page_compact(host[0], host[1], host[3])
            host[0], host[3] = t, r
            for x in state:
                for a, b in copies:
                    x[b] = x[a]
            assert np.array_equal(table.cpu().numpy(), t) and np.array_equal(refs.cpu().numpy(), r)
            assert all(np.array_equal(x, y) for x, y in zip(raw(), state))


@pytest.mark.parametrize("q", [3, 50])
def test_offsets_past_32_bits(sv, q):
    """Pages that lie more than 2^32 bytes into their arrays: append, attention, a copy of a shared page, a move."""
    torch = torch_mod()
    Hkv, D, page, block, pages = 8, 128, 64, 32, 70000  # 4.6 GB each
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("not enough memory")
    kp, vp = (torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ke, ve = (torch.full((pages, Hkv, page // block), 120, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Attn([q], [150], G=4, Hkv=Hkv, D=D, page=page, block=block, append=True, seed=1, lead=0, trail=0)
    c.table[:, :3] = [0, 1, 2]
    ids = [pages - 1, pages - 2, pages - 5]
    codes = np.full((3, Hkv, page, D), 0x38, np.uint8)
    c.codes, c.exps = [codes.copy(), codes.copy()], [np.full((3, Hkv, 2), 120, np.uint8) for _ in range(2)]
    rng = np.random.default_rng(0)
    for x in c.codes:
        x[:] = rng.integers(0, 0x60, x.shape)
    c.pages = 3
    for n, i in enumerate(ids):
        kp.view(torch.uint8)[i], vp.view(torch.uint8)[i] = (torch.from_numpy(x[n]).cuda() for x in c.codes)
    (ref, A, W, S), state = c.reference()
    table, lens, refs = i32([ids + [0]]), i32([150]), torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[ids] = 1
    o = torch.empty(q, 4 * Hkv, D, dtype=torch.float32, device="cuda")
    sv.spec_paged_attn8(c.q.cuda(), kp, vp, ke, ve, table, i32([0, q]), lens, o, max_q=q, k_new=c.new[0].cuda(), v_new=c.new[1].cuda())
    check(np64(o), ref, A, W, S, D, 150, "f32")
    got = lambda x, at: x.view(torch.uint8)[at].cpu().numpy()  # noqa: E731
    for x, want in zip((kp, vp, ke, ve), state):
        assert np.array_equal(got(x, ids), want)
    # a second holder of the last page: the row's own copy is the lowest free page, then everything moves down
    refs[ids[2]] = 2
    held = i32([3])
    sv.spec_page_fork(table, held, lens, refs, i32([0]), page_size=page, grow=i32([1]), caches=[kp, vp, ke, ve])
    assert table[0, :3].tolist() == ids[:2] + [0] and np.array_equal(got(kp, 0), state[0][2])
    moved = torch.zeros(pages, dtype=torch.int32, device="cuda")
    sv.spec_page_compact(table, held, refs, caches=[kp, vp, ke, ve], moved=moved)
    assert table[0, :3].tolist() == [3, 2, 0] and moved[ids[2]] == 1
    for x, want in zip((kp, vp, ke, ve), state):
        assert np.array_equal(got(x, [3, 2, 0]), want[[0, 1, 2]])
