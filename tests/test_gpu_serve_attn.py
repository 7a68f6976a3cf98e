"""GPU parity of spec_paged_attn and spec_prefill_attn against the float64 oracle, element by element.

Tolerance of an output element, derived: with A = sum_t p_t |v_t| and r the largest relative error of a
probability, |o - exact| <= 2 r A (the numerator's and the normaliser's share) plus the output's own
rounding.  r: the score is a D-term fp32 sum, off by at most (D + 8) 2^-24 S with S the largest
scale * sum |q k| (S enters absolutely: it sits in an exponent), plus 2^-20 for 2^x and the running
rescales, plus half an ulp of bf16 (2^-8 relative; P is rounded, its sum is not) where K/V are bf16.
The P.V and l sums over L keys add L 2^-24 A each.  Slots past kv_len, free pages and pages before the
window hold NaN; rows of no sequence hold a sentinel that must survive.
"""

import numpy as np
import pytest

from oracle import serve as os_

from .helpers import torch_mod

pytestmark = pytest.mark.gpu

SENTINEL = 7.5


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def tolerance(ref, A, S, D, L, kv_dtype, o_dtype):
    r = (D + 8) * 2.0 ** -24 * S + 2.0 ** -20
    tol = (2 * r + 2 * L * 2.0 ** -24) * A
    if kv_dtype == "bf16":
        tol = tol + 2.0 ** -8 * A
    return tol + (2.0 ** -8 if o_dtype == "bf16" else 2.0 ** -24) * np.abs(ref) + 1e-30


def check(o, ref, A, S, D, L, kv_dtype, o_dtype, what=""):
    assert np.all(np.isfinite(o)), f"{what}: non-finite output"
    over = np.abs(o - ref) / tolerance(ref, A, S, D, L, kv_dtype, o_dtype)
    assert over.max(initial=0) <= 1, f"{what}: {over.max():.3g} times the bound at {np.unravel_index(over.argmax(), over.shape)}"


def dt(name):
    torch = torch_mod()
    return torch.bfloat16 if name == "bf16" else torch.float32


def np64(t):
    return t.detach().double().cpu().numpy()


class Paged:
    """Seeded inputs on the device; every place that must not be read holds NaN."""

    def __init__(self, q_len, kv_len, Hq, Hkv, D, page, dtype="bf16", window=0, seed=0, lead=0, trail=3, layout="hnd",
                 append=False, extra_pages=3):
        torch = torch_mod()
        g = torch.Generator().manual_seed(seed)
        self.page, self.D, self.dtype, self.window, self.append = page, D, dtype, window, append
        self.Hkv, self.B = Hkv, len(q_len)
        self.start = np.cumsum([lead] + list(q_len)).astype(np.int32)
        self.kv_len = np.array(kv_len, dtype=np.int32)
        T = self.start[-1] + trail
        per = [-(-n // page) for n in kv_len]
        pages = sum(per) + extra_pages
        order = torch.randperm(pages, generator=g).numpy()
        self.table = np.full((self.B, max(max(per), 1)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        norm = lambda *s: torch.randn(*s, generator=g).to(dt(dtype))  # noqa: E731
        self.q = norm(T, Hq, D)
        self.q[:lead] = float("nan")
        self.q[self.start[-1]:] = float("nan")
        kp = torch.full((pages, Hkv, page, D), float("nan"), dtype=dt(dtype))
        vp = kp.clone()
        for b in range(self.B):
            n = int(q_len[b])
            lo = max(0, int(kv_len[b]) - n + 1 - window) if window else 0
            hi = int(kv_len[b]) - n if append else int(kv_len[b])
            if n == 0:
                continue
            for t in range(lo, hi):
                kp[self.table[b, t // page], :, t % page] = norm(Hkv, D)
                vp[self.table[b, t // page], :, t % page] = norm(Hkv, D)
            if window:
                self.table[b, :lo // page] = -5  # given back
        self.k_new = norm(T, Hkv, D) if append else None
        self.v_new = norm(T, Hkv, D) if append else None
        if append:
            for x in (self.k_new, self.v_new):
                x[:lead] = float("nan")
                x[self.start[-1]:] = float("nan")
        if layout == "nhd":  # tokens before heads, in a buffer with K and V of a page side by side
            both = torch.empty((pages, page, 2, Hkv, D), dtype=dt(dtype))
            both[:, :, 0] = kp.permute(0, 2, 1, 3)
            both[:, :, 1] = vp.permute(0, 2, 1, 3)
            both = both.cuda()
            self.k, self.v = both[:, :, 0].permute(0, 2, 1, 3), both[:, :, 1].permute(0, 2, 1, 3)
        else:
            self.k, self.v = kp.cuda(), vp.cuda()
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        self.d_q = self.q.cuda()
        self.d_table, self.d_start, self.d_len = dev(self.table), dev(self.start), dev(self.kv_len)
        self.d_new = {} if not append else dict(k_new=self.k_new.cuda(), v_new=self.v_new.cuda())
        self.max_q = max(max(q_len), 1)

    def oracle(self):
        kp, vp = np64(self.k), np64(self.v)
        if self.append:
            kp, vp = os_.append_pages(kp, vp, self.table, self.start, self.kv_len, np64(self.k_new), np64(self.v_new))
        return os_.paged_attn(np64(self.q), kp, vp, self.table, self.start, self.kv_len, self.window), kp, vp

    def run(self, sv, o_dtype="f32", o=None, max_q=None, **kw):
        torch = torch_mod()
        if o is None:
            o = torch.full(self.q.shape, SENTINEL, dtype=dt(o_dtype), device="cuda")
        max_q = max_q or self.max_q
        ws = torch.full((sv.spec_paged_attn_workspace(self.d_q, self.k, self.d_table, o, max_q=max_q),), 255,
                        dtype=torch.uint8, device="cuda")
        sv.spec_paged_attn(self.d_q, self.k, self.v, self.d_table, self.d_start, self.d_len, o, max_q=max_q,
                           window=self.window, workspace=ws, **self.d_new, **kw)
        torch.cuda.synchronize()
        return np64(o), sv.read_status(ws)

    def verify(self, sv, o_dtype="f32", what="", **kw):
        (ref, A, S), kp, vp = self.oracle()
        o, st = self.run(sv, o_dtype, **kw)
        r0, r1 = self.start[0], self.start[-1]
        assert st == 0
        check(o[r0:r1], ref[r0:r1], A[r0:r1], S, self.D, int(self.kv_len.max()), self.dtype, o_dtype, what)
        assert np.all(o[:r0] == SENTINEL) and np.all(o[r1:] == SENTINEL)
        # the pages: appended rows bit for bit, everything else as it was
        assert np.array_equal(np64(self.k), kp, equal_nan=True) and np.array_equal(np64(self.v), vp, equal_nan=True)
        return o


SMALL = [  # up to 32 query rows per kv head
    ([1], [1], 4, 1, 16),
    ([1], [300], 32, 8, 16),
    ([5, 5, 5], [1500, 2113, 777], 32, 8, 64),
    ([1, 0, 3, 8, 0, 2], [640, 9, 3, 900, 50, 130], 8, 2, 32),
    ([7, 1], [1000, 2047], 3, 3, 128),
    ([1, 1], [4000, 17], 32, 1, 7),
    ([4], [5000], 8, 1, 24),
    ([2, 1, 2], [33, 1, 128], 16, 1, 1),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("case", range(len(SMALL)))
def test_small_chunks(sv, case, append, D):
    q_len, kv_len, Hq, Hkv, page = SMALL[case]
    Paged(q_len, kv_len, Hq, Hkv, D, page, append=append, seed=case).verify(sv, what=f"case {case}")


LARGE = [  # more rows: the tiled kernels
    ([40], [40], 4, 1, 16),
    ([70, 0, 9, 130], [70, 5, 600, 1300], 8, 2, 64),
    ([33, 1, 64, 2], [1700, 900, 64, 3], 12, 4, 24),
    ([300], [420], 2, 2, 128),
    ([130, 200], [1100, 200], 6, 2, 32),
    ([9, 10], [2600, 2000], 32, 2, 256),
    ([257], [1500], 1, 1, 5),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("case", range(len(LARGE)))
def test_large_chunks(sv, case, append, D):
    q_len, kv_len, Hq, Hkv, page = LARGE[case]
    Paged(q_len, kv_len, Hq, Hkv, D, page, append=append, seed=20 + case).verify(sv, what=f"case {case}")


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,D,page", [
    ([1], [1], 1, 1, 64, 16), ([1, 5, 0, 33], [90, 300, 4, 700], 4, 1, 64, 16), ([80, 3], [500, 60], 8, 4, 128, 48),
    ([2], [3000], 4, 2, 128, 64)])
def test_fp32_cache(sv, q_len, kv_len, Hq, Hkv, D, page, append):
    Paged(q_len, kv_len, Hq, Hkv, D, page, dtype="f32", append=append, seed=40).verify(sv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
@pytest.mark.parametrize("q_len,kv_len", [([1, 4, 0, 3], [900, 300, 20, 3]), ([50, 1, 129], [700, 800, 129])])
def test_window(sv, q_len, kv_len, window, dtype):
    """Table entries and pages wholly before the window are never looked at."""
    Paged(q_len, kv_len, 8, 2, 64, 16, dtype=dtype, window=window, append=True, seed=50 + window).verify(sv)


@pytest.mark.parametrize("q_len,kv_len", [([3, 5], [200, 900]), ([40, 20], [300, 900])])
def test_layouts_and_bf16_output(sv, q_len, kv_len):
    """Token-major pages with K and V side by side, leading rows, a strided bf16 output."""
    torch = torch_mod()
    p = Paged(q_len, kv_len, 8, 2, 128, 32, layout="nhd", append=True, lead=5, seed=60)
    p.verify(sv, "bf16")
    (ref, A, S), _, _ = p.oracle()
    wide = torch.full((p.q.shape[0], 8, 131), SENTINEL, dtype=torch.bfloat16, device="cuda")
    o, st = p.run(sv, o=wide[:, :, 1:129])
    assert st == 0
    r0, r1 = p.start[0], p.start[-1]
    check(o[r0:r1], ref[r0:r1], A[r0:r1], S, 128, 900, "bf16", "bf16")
    w = np64(wide)
    assert np.all(w[:, :, 0] == SENTINEL) and np.all(w[:, :, 129:] == SENTINEL)
    # a q whose rows are spread out
    big = torch.full((p.q.shape[0], 3, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 1] = p.d_q
    p.d_q = big[:, 1]
    p.verify(sv, "bf16")


@pytest.mark.parametrize("q,page", [(1, 16), (20, 16)])
def test_many_sequences(sv, q, page):
    rng = np.random.default_rng(7)
    B = 700
    q_len = [int(x) for x in rng.integers(0, q + 1, B)]
    q_len[0] = q
    kv_len = [n + int(x) for n, x in zip(q_len, rng.integers(0, 40, B))]
    kv_len[5] = q_len[5] + 600
    Paged(q_len, kv_len, 4, 2, 64, page, append=True, seed=70).verify(sv)


@pytest.mark.parametrize("q", [1, 40])
def test_most_sequences(sv, q):
    """4096 sequences, most of them resting, and a bound on the chunk lengths that is far too wide."""
    rng = np.random.default_rng(8)
    q_len = [0] * 4096
    for b in rng.integers(0, 4096, 150):
        q_len[b] = int(rng.integers(1, q + 1))
    q_len[0] = q_len[4095] = q
    kv_len = [n + int(x) for n, x in zip(q_len, rng.integers(0, 3, 4096))]
    p = Paged(q_len, kv_len, 1, 1, 64, 4, seed=75)
    p.verify(sv)
    p.verify(sv, max_q=10 ** 6)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_cut_tile_beside_uneven_rounds(sv, page, D):
    # a long sequence whose tiles are cut, the first piece on CTA 0 early, and 900 small tiles that do not fill
    # their last round: the CTAs that go without leave the cut tiles' records alone
    case = Paged([64] + [64] * 450, [16384] + [64] * 450, 8, 2, D, page, append=True, seed=41)
    first = case.verify(sv)
    for _ in range(4):
        o, st = case.run(sv)
        assert st == 0 and np.array_equal(o, first, equal_nan=True)


@pytest.mark.parametrize("G", [1, 4, 16])
@pytest.mark.parametrize("rows", [16, 17, 32, 33, 128, 129, 256, 257])
def test_row_boundaries(sv, rows, G):
    """One row more or less than each tile of the kernels holds."""
    n = -(-rows // G)
    Paged([n, 1], [n + 200, 77], G, 1, 64, 32, append=True, seed=rows + G).verify(sv)


@pytest.mark.parametrize("q_len", [[1, 3], [50, 20]])
def test_shared_prefix_and_large_pages(sv, q_len):
    """Two sequences whose first pages are the same ones; a page much longer than the sequences."""
    torch = torch_mod()
    p = Paged(q_len, [400, 380], 8, 2, 64, 64, seed=77)
    p.table[1, :4] = p.table[0, :4]
    p.d_table = torch.from_numpy(p.table).cuda()
    p.verify(sv)
    Paged(q_len, [400, 380], 8, 2, 64, 1000, append=True, seed=78).verify(sv)


def test_binding_refusals(sv):
    torch = torch_mod()
    p = Paged([3], [40], 4, 2, 64, 16, seed=79)
    o = torch.empty(p.q.shape, device="cuda")
    call = lambda **kw: sv.spec_paged_attn(**dict(dict(q=p.d_q, k_pages=p.k, v_pages=p.v, page_table=p.d_table,  # noqa: E731
                                                      q_start=p.d_start, kv_len=p.d_len, o=o, max_q=3), **kw))
    with pytest.raises(ValueError):
        call(kv_len=p.d_len.long())
    with pytest.raises(ValueError):
        call(kv_len=p.d_len.cpu())
    with pytest.raises(ValueError):
        call(workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(q=p.d_q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(TypeError):
        call(q=p.d_q.half())
    for bad in (dict(q=p.d_q.float()), dict(window=-1), dict(max_q=0), dict(scale=float("inf"))):
        with pytest.raises(sv.SpecError):
            call(**bad)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    with pytest.raises(sv.SpecError):
        call(workspace=ws[8:])
    call(workspace=ws)
    empty = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    zeros = torch.zeros(2, dtype=torch.int32, device="cuda")
    sv.spec_paged_attn(empty, p.k, p.v, p.d_table, zeros, p.d_len, empty, max_q=1)
    sv.spec_prefill_attn(empty, empty, empty, zeros, empty)
    torch.cuda.synchronize()


@pytest.mark.parametrize("cols", [0, 200])
@pytest.mark.parametrize("q_len", [[2, 3, 1, 4], [40, 3, 1, 20]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_data_is_flagged_and_contained(sv, q_len, dtype, cols):
    """cols: table columns beyond what the sequences need (a larger capacity takes other kernels)."""
    torch = torch_mod()
    kv_len = [300, 200, 500, 250]
    p = Paged(q_len, kv_len, 8, 2, 64, 16, dtype=dtype, append=True, seed=80)
    p.table = np.concatenate([p.table, np.full((4, cols), -9, dtype=np.int32)], axis=1)
    p.d_table = torch.from_numpy(p.table).cuda()
    capacity = 16 * p.table.shape[1]
    (ref, A, S), kp, vp = p.oracle()
    rows = lambda b: slice(p.start[b], p.start[b + 1])  # noqa: E731
    good = p.run(sv)[0]
    check(good[rows(0)], ref[rows(0)], A[rows(0)], S, 64, 500, dtype, "f32")
    # a length above the table's capacity, and one below the chunk's
    for bad in (capacity + 1, q_len[1] - 1, -4):
        p.d_len[1] = bad
        before = np64(p.k)
        o, st = p.run(sv)
        assert st == sv.SPEC_STATUS_BAD_KV_LEN
        assert np.all(o[rows(1)] == 0)
        assert np.array_equal(np64(p.k), before, equal_nan=True)
        for b in (0, 2, 3):
            assert np.max(np.abs(o[rows(b)] - good[rows(b)])) < 1e-2
    p.d_len[1] = 200
    # the same with no append, where a call has the least kernels
    new, p.d_new = p.d_new, {}
    p.d_len[1] = capacity + 1
    o, st = p.run(sv)
    assert st == sv.SPEC_STATUS_BAD_KV_LEN and np.all(o[rows(1)] == 0)
    p.d_len[1] = 200
    p.d_table[2, 3] = -1
    o, st = p.run(sv)
    assert st == sv.SPEC_STATUS_BAD_PAGE and np.all(np.isfinite(o[p.start[0]:p.start[-1]]))
    p.d_table[2, 3] = int(p.table[2, 3])
    p.d_new = new
    # page ids out of range
    for bad in (-1, p.k.shape[0], 2 ** 31 - 1):
        p.d_table[2, 3] = bad
        o, st = p.run(sv)
        assert st == sv.SPEC_STATUS_BAD_PAGE
        assert np.all(np.isfinite(o[p.start[0]:p.start[-1]]))
        for b in (0, 1, 3):
            assert np.max(np.abs(o[rows(b)] - good[rows(b)])) < 1e-2
    p.d_table[2, 3] = int(p.table[2, 3])
    # chunk ranges out of order, outside q, or above max_q
    T = p.q.shape[0]
    for at, val in ((4, T + 1), (4, int(p.start[3]) - 1), (0, -2)):
        s = p.start.copy()
        s[at] = val
        p.d_start = torch.from_numpy(s).cuda()
        o, st = p.run(sv)
        assert st == sv.SPEC_STATUS_BAD_RANGE
        hit = 3 if at == 4 else 0
        assert np.all(o[rows(hit)] == SENTINEL)
        for b in (1, 2):
            assert np.max(np.abs(o[rows(b)] - good[rows(b)])) < 1e-2
    p.d_start = torch.from_numpy(np.array([0, T, 0, T, 0], dtype=np.int32)).cuda()  # overlapping
    p.d_len[:] = 500
    p.d_new = {}
    p.table[:] = 0
    p.d_table[:] = 0
    o, st = p.run(sv, max_q=T)
    assert st & sv.SPEC_STATUS_BAD_RANGE
    # and the next call is clean again
    p = Paged(q_len, kv_len, 8, 2, 64, 16, dtype=dtype, append=True, seed=81)
    p.verify(sv)


@pytest.mark.parametrize("q_len", [[1, 1], [30, 12]])
def test_offsets_past_32_bits(sv, q_len):
    """Pages whose element offsets pass 2^31."""
    torch = torch_mod()
    p = Paged(q_len, [400, 90], 8, 2, 128, 16, seed=90)
    n, old = p.k.shape[0], p.k.shape
    pages = 2 ** 31 // (2 * 16 * 128) + 2 * n
    shift = pages - n
    big = []
    for x in (p.k, p.v):
        y = torch.zeros((pages, *old[1:]), dtype=torch.bfloat16, device="cuda")
        y[shift:] = x
        big.append(y)
    (ref, A, S), _, _ = p.oracle()
    p.k, p.v = big
    p.d_table = torch.where(p.d_table >= 0, p.d_table + shift, p.d_table)
    o, st = p.run(sv)
    assert st == 0
    check(o[:p.start[-1]], ref[:p.start[-1]], A[:p.start[-1]], S, 128, 400, "bf16", "f32")


@pytest.mark.parametrize("q_len,other", [([1, 2], [2, 0]), ([20, 1], [3, 18])])
def test_graph_replay_reads_new_lengths(sv, q_len, other):
    torch = torch_mod()
    a = Paged(q_len, [300, 150], 8, 2, 64, 16, append=True, seed=100)
    b = Paged(other, [200, 310], 8, 2, 64, 16, append=True, seed=101, trail=3 + sum(q_len) - sum(other))
    n = max(a.k.shape[0], b.k.shape[0])
    cols = max(a.table.shape[1], b.table.shape[1])
    k = torch.zeros((n, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    v, table = torch.zeros_like(k), torch.zeros((2, cols), dtype=torch.int32, device="cuda")
    q, kn, vn = torch.empty_like(a.d_q), torch.empty_like(a.d_new["k_new"]), torch.empty_like(a.d_new["v_new"])
    start, lens, o = torch.empty_like(a.d_start), torch.empty_like(a.d_len), torch.empty(q.shape, device="cuda")
    max_q = max(*q_len, *other)
    ws = torch.empty(sv.spec_paged_attn_workspace(q, k, table, o, max_q=max_q), dtype=torch.uint8, device="cuda")

    def load(x):
        k[:x.k.shape[0]] = x.k
        v[:x.v.shape[0]] = x.v
        table[:, :x.table.shape[1]] = x.d_table
        for d, s in ((q, x.d_q), (kn, x.d_new["k_new"]), (vn, x.d_new["v_new"]), (start, x.d_start), (lens, x.d_len)):
            d.copy_(s)
        o.fill_(SENTINEL)

    def call():
        sv.spec_paged_attn(q, k, v, table, start, lens, o, max_q=max_q, k_new=kn, v_new=vn,
                           workspace=ws)

    load(a)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in (b, a, b):
        (ref, A, S), kp, _ = x.oracle()
        load(x)
        g.replay()
        torch.cuda.synchronize()
        r = x.start[-1]
        got = np64(o)
        check(got[:r], ref[:r], A[:r], S, 64, 310, "bf16", "f32")
        assert np.all(got[r:] == SENTINEL) and sv.read_status(ws) == 0


@pytest.mark.parametrize("q_len", [[4, 1], [60, 9]])
def test_streams_and_determinism(sv, q_len):
    """Two calls at once on two streams (own workspaces); repeated calls give the same bits."""
    torch = torch_mod()
    ps = [Paged(q_len, [2000, 700], 8, 2, 128, 16, seed=110 + i) for i in range(2)]
    want = [p.run(sv)[0] for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(3):
        outs = []
        for p, s in zip(ps, streams):
            o = torch.full(p.q.shape, SENTINEL, device="cuda")
            torch.cuda.synchronize()
            outs.append(o)
        for p, s, o in zip(ps, streams, outs):
            sv.spec_paged_attn(p.d_q, p.k, p.v, p.d_table, p.d_start, p.d_len, o, max_q=p.max_q, stream=s)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert np.array_equal(np64(o), w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,Hq,Hkv,lens,window", [
    (64, 4, 1, [7, 130, 1, 0, 65], 0), (128, 8, 2, [300], 0), (128, 6, 2, [1, 1, 2, 257], 0),
    (64, 8, 8, [129, 400], 64), (128, 32, 4, [20, 0, 33], 1), (64, 32, 1, [90], 0), (128, 2, 1, [700, 3, 0, 300], 0),
    (64, 4, 2, [900], 200)])
def test_prefill(sv, dtype, D, Hq, Hkv, lens, window):
    torch = torch_mod()
    g = torch.Generator().manual_seed(sum(lens) + D)
    lead, T = 2, 2 + sum(lens) + 4
    start = np.cumsum([lead] + lens).astype(np.int32)
    q, k, v = (torch.randn(T, h, D, generator=g).to(dt(dtype)) for h in (Hq, Hkv, Hkv))
    for x in (q, k, v):
        x[:lead] = float("nan")
        x[start[-1]:] = float("nan")
    ref, A, S = os_.prefill_attn(np64(q), np64(k), np64(v), start, window)
    for o_dtype in ("f32", "bf16"):
        o = torch.full((T, Hq, D), SENTINEL, dtype=dt(o_dtype), device="cuda")
        kv = torch.stack([k, v], dim=1).cuda()  # K and V rows side by side: strided views
        dq, ds = q.cuda(), torch.from_numpy(start).cuda()
        ws = torch.empty(sv.spec_prefill_attn_workspace(dq, kv[:, 0], ds, o), dtype=torch.uint8, device="cuda")
        sv.spec_prefill_attn(dq, kv[:, 0], kv[:, 1], ds, o, window=window, workspace=ws)
        torch.cuda.synchronize()
        assert sv.read_status(ws) == 0
        got, r = np64(o), slice(lead, start[-1])
        check(got[r], ref[r], A[r], S, D, max(lens), dtype, o_dtype)
        assert np.all(got[:lead] == SENTINEL) and np.all(got[start[-1]:] == SENTINEL)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [300, 1500])
def test_prefill_bad_ranges(sv, T, dtype):
    """Sequences whose range is out of order have no output; their neighbours' is right."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(T, h, 64, generator=g).to(dt(dtype)) for h in (2, 1, 1))
    good = np.array([0, 90, 200, 260], dtype=np.int32)
    ref, A, S = os_.prefill_attn(np64(q)[:260], np64(k)[:260], np64(v)[:260], good)
    for bad, rows, none in (([0, 90, 200, T + 1], slice(0, 200), slice(200, T)),
                            ([0, 90, 40, 260], slice(0, 40), slice(260, T)),
                            ([-1, 90, 200, 260], slice(90, 260), slice(0, 90))):
        o = torch.full((T, 2, 64), SENTINEL, device="cuda")
        start = torch.tensor(bad, dtype=torch.int32, device="cuda")
        dq, dk = q.cuda(), k.cuda()
        ws = torch.empty(sv.spec_prefill_attn_workspace(dq, dk, start, o), dtype=torch.uint8, device="cuda")
        sv.spec_prefill_attn(dq, dk, v.cuda(), start, o, workspace=ws)
        torch.cuda.synchronize()
        got = np64(o)
        assert sv.read_status(ws) == sv.SPEC_STATUS_BAD_RANGE
        check(got[rows], ref[rows], A[rows], S, 64, 200, dtype, "f32")
        assert np.all(got[none] == SENTINEL)


def test_prefill_neighbours_do_not_leak(sv):
    """A sequence of NaN and infinities leaves its neighbours alone."""
    torch = torch_mod()
    lens = [50, 40, 70]
    start = np.cumsum([0] + lens).astype(np.int32)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(160, h, 64, generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    ref, A, S = os_.prefill_attn(np64(q), np64(k), np64(v), start)
    k[50:90], v[50:90:2], v[51:90:2] = float("nan"), float("inf"), float("nan")
    o = torch.empty((160, 4, 64), device="cuda")
    sv.spec_prefill_attn(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(start).cuda(), o)
    got = np64(o)
    for r in (slice(0, 50), slice(90, 160)):
        check(got[r], ref[r], A[r], S, 64, 70, "bf16", "f32")


def test_large_scores_and_scale(sv):
    """Scores far beyond the exponent's range, with an explicit scale: the softmax is a maximum."""
    torch = torch_mod()
    p = Paged([3, 40], [200, 300], 4, 1, 64, 16, seed=130)
    p.d_q.mul_(64)
    p.q.mul_(64)
    kp, vp = np64(p.k), np64(p.v)
    ref, A, S = os_.paged_attn(np64(p.q), kp, vp, p.table, p.start, p.kv_len, scale=2.0)
    o, st = p.run(sv, scale=2.0)
    assert st == 0
    r = p.start[-1]
    # S is in the thousands here, so the bound's absolute error of a score is about 0.1
    check(o[:r], ref[:r], A[:r], S, 64, 300, "bf16", "f32")


@pytest.mark.parametrize("q_len", [[2], [60]])
@pytest.mark.parametrize("growth", [0.02, 0.2, -0.2])
def test_rising_scores(sv, q_len, growth):
    """Scores that rise (or fall) along the keys, so that the running reference lags behind the maximum
    by a few powers of two, or has to move in every tile."""
    torch = torch_mod()
    p = Paged(q_len, [1500], 4, 2, 64, 64, seed=140)
    k = p.k.float().cpu()
    u = torch.randn(64, generator=torch.Generator().manual_seed(1))
    u /= u.norm()
    for t in range(1500):
        k[p.table[0, t // 64], :, t % 64] = 0.2 * k[p.table[0, t // 64], :, t % 64] + growth * t * u
    p.k = k.to(torch.bfloat16).cuda()
    p.q = (p.q.float() * 0.1 + 4 * u).to(torch.bfloat16)
    p.d_q = p.q.cuda()
    (ref, A, S), _, _ = p.oracle()
    o, st = p.run(sv)
    assert st == 0
    r = p.start[-1]
    check(o[:r], ref[:r], A[:r], S, 64, 1500, "bf16", "f32")


def test_mixed_lists_agree_with_verify_attn(sv):
    """The paged call on pages that tile a dense cache gives spec_verify_attn's answer."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(6)
    B, nq, Hq, Hkv, D, L = 3, 5, 8, 2, 128, 512
    k, v = (torch.randn(B, Hkv, L, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(B, nq, Hq, D, generator=g).to(torch.bfloat16).cuda()
    lens = torch.tensor([512, 77, 300], dtype=torch.int32, device="cuda")
    dense = sv.spec_verify_attn(q, k, v, lens, torch.empty(q.shape, device="cuda"))
    page = 32
    pages = [x.view(B, Hkv, L // page, page, D).permute(0, 2, 1, 3, 4).reshape(-1, Hkv, page, D).contiguous()
             for x in (k, v)]
    table = torch.arange(B * L // page, dtype=torch.int32, device="cuda").view(B, -1)
    start = torch.arange(0, B * nq + 1, nq, dtype=torch.int32, device="cuda")
    o = sv.spec_paged_attn(q.view(-1, Hq, D), *pages, table, start, lens, torch.empty((B * nq, Hq, D), device="cuda"),
                           max_q=nq)
    # two evaluations of the same bf16 products, each with P rounded to bf16 against its own maximum
    assert float((o.view_as(dense) - dense).abs().max()) <= 2 * 2.0 ** -8 * float(v.abs().max())
