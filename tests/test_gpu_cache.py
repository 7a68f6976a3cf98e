"""GPU parity of spec_rotary and spec_kv8_append against the float64 oracle.

Rotary, derived: sine and cosine of a phase rounded to 24 bits (off by at most 2^-25 of half a turn's range,
pi 2^-24 in all) and CUDA's sincospi (2 ulp, 2^-22 of 1); times the amplitude (2^-24) and two products and a sum in
fp32 (2^-24 each): below (|a| + |b|) * amplitude * 2^-20.5 < 2^-20 (|a| + |b|) amplitude; then half a step of the
output's type.  The append is exact: codes and bytes are compared bit for bit."""

import math

import numpy as np
import pytest

from oracle import cache as oc

from .helpers import torch_mod

pytestmark = pytest.mark.gpu

SENTINEL = 7.5


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def dt(name):
    torch = torch_mod()
    return torch.bfloat16 if name == "bf16" else torch.float32


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    torch = torch_mod()
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


# ------------------------------------------------------------------------------ rotary
def rotary_bound(x, ref, half, pairs, amplitude, dtype):
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    s = (np.abs(a) + np.abs(b)) * amplitude * 2.0 ** -20
    tol = np.zeros_like(x)
    if pairs:
        tol[..., 0:2 * half:2] = tol[..., 1:2 * half:2] = s
    else:
        tol[..., :half] = tol[..., half:2 * half] = s
    return tol + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(ref) * (np.arange(x.shape[-1]) < 2 * half)


def turns_to_frequencies(steps):
    return steps.cpu().numpy().astype(np.longdouble) / np.longdouble(2.0) ** 64 * 2 * np.longdouble(math.pi)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,far", [
    (1, 1, 1, 8, 2, "bf16", 10), (5, 4, 1, 64, 64, "f32", 500), (3, 32, 8, 128, 128, "bf16", 32768),
    (17, 5, 3, 128, 116, "bf16", 1 << 20), (9, 2, 2, 64, 20, "f32", 1 << 24), (700, 3, 1, 128, 32, "bf16", 2 ** 31 - 1),
    (1300, 2, 1, 64, 64, "f32", 100000), (5000, 4, 2, 128, 64, "bf16", 4096), (4, 1, 1, 1024, 1024, "bf16", 1000),
    (4, 2, 0, 256, 256, "f32", 1000), (6, 0, 2, 80, 48, "bf16", 1000), (9, 2, 2, 64, 24, "bf16", 1000), (9, 2, 2, 64, 10, "f32", 1000),
    (3, 2, 1, 1024, 1022, "bf16", 1000), (30, 7, 5, 64, 6, "bf16", 1000)])
def test_rotary_parity(sv, T, Hq, Hkv, D, rot, dtype, far, pairs):
    torch = torch_mod()
    rng = np.random.default_rng(T + D + rot)
    pos = rng.integers(0, far, T)
    pos[0], pos[-1] = -3, far - 1 if far - 1 < 2 ** 31 else 2 ** 31 - 1
    steps, amp = sv.spec_rotary_steps(rot, 10000.0, kind=sv.SPEC_ROTARY_YARN, factor=4.0, length=4096.0)
    make = lambda H: torch.from_numpy(rng.standard_normal((T, H, D))).to(dt(dtype)).cuda() if H else None  # noqa: E731
    q, k = make(Hq), make(Hkv)
    f = turns_to_frequencies(steps)
    kw = dict(positions=i32(pos), layout=sv.SPEC_ROTARY_PAIRS if pairs else sv.SPEC_ROTARY_HALF, amplitude=amp)
    before = [None if x is None else np64(x) for x in (q, k)]
    apart = [None if x is None else torch.full_like(x, SENTINEL) for x in (q, k)]
    sv.spec_rotary(q, k, steps, q_out=apart[0], k_out=apart[1], **kw)
    for x, y, x0 in zip((q, k), apart, before):
        if x is None:
            continue
        assert np.array_equal(np64(x), x0)
        ref = oc.rotary(x0, pos, f, pairs, amp)
        assert np.all(np.abs(np64(y) - ref) <= rotary_bound(x0, ref, rot // 2, pairs, amp, dtype))
        assert np.array_equal(np64(y)[..., rot:], x0[..., rot:])
    # in place, the same bits
    sv.spec_rotary(q, k, steps, **kw)
    for x, y in zip((q, k), apart):
        assert x is None or torch.equal(x, y)


def test_rotary_inverse_and_gradient(sv):
    """The way back undoes the way there, and is its gradient: for L = sum(w * rotary(x)), dL/dx = inverse(w)."""
    torch = torch_mod()
    rng = np.random.default_rng(8)
    x, w = (torch.from_numpy(rng.standard_normal((11, 3, 64))).float().cuda() for _ in range(2))
    steps, _ = sv.spec_rotary_steps(48)
    kw = dict(positions=i32(rng.integers(0, 5000, 11)), layout=sv.SPEC_ROTARY_PAIRS)
    y, _ = sv.spec_rotary(x, None, steps, q_out=torch.empty_like(x), **kw)
    back, _ = sv.spec_rotary(y, None, steps, q_out=torch.empty_like(x), inverse=True, **kw)
    # two turns, each within 2^-20 (|a| + |b|)
    assert np.all(np.abs(np64(back) - np64(x)) <= 2.0 ** -18 * np.abs(np64(x)).max())
    g, _ = sv.spec_rotary(w, None, steps, q_out=torch.empty_like(x), inverse=True, **kw)
    f = turns_to_frequencies(steps)
    pos = kw["positions"].cpu().numpy()
    ref = np.zeros(x.shape)
    basis = np.eye(64)
    for t in range(11):
        turned = oc.rotary(basis[:, None, :], [pos[t]] * 64, f, True)[:, 0]  # row i: where value i goes
        ref[t] = np64(w)[t] @ turned.T
    assert np.all(np.abs(np64(g) - ref) <= rotary_bound(np64(w), ref, 24, True, 1.0, "f32") + 1e-12)
    h, d = 2.0 ** -7, torch.from_numpy(rng.standard_normal(x.shape)).float().cuda()
    up, _ = sv.spec_rotary(x + h * d, None, steps, q_out=torch.empty_like(x), **kw)
    down, _ = sv.spec_rotary(x - h * d, None, steps, q_out=torch.empty_like(x), **kw)
    slope = float(((up.double() - down.double()) * w.double()).sum() / (2 * h))
    # the map is linear: what differs is 2113 roundings of at most 2^-20 * 10 over 2 h = 2^-6, and as many of w's
    assert abs(slope - float((g.double() * d.double()).sum())) <= 2112 * 10 * 4 * 2.0 ** -20 / 2.0 ** -6


@pytest.mark.parametrize("B,T", [(1, 1), (3, 40), (4096, 5000)])
def test_rotary_of_a_ragged_batch(sv, B, T):
    torch = torch_mod()
    rng = np.random.default_rng(B)
    cuts = np.sort(rng.integers(2 if T > 5 else 0, T - 1 if T > 5 else T + 1, B - 1))
    start = np.concatenate(([2 if T > 5 else 0], cuts, [T - 1 if T > 5 else T])).astype(np.int32)
    n = np.diff(start)
    lens = n + rng.integers(0, 1000, B)
    x = torch.from_numpy(rng.standard_normal((T, 2, 64))).float().cuda()
    x0 = np64(x)
    steps, _ = sv.spec_rotary_steps(64)
    ws = torch.full((sv.spec_rotary_workspace(x, None, steps),), 255, dtype=torch.uint8, device="cuda")
    sv.spec_rotary(x, None, steps, q_start=i32(start), kv_len=i32(lens), workspace=ws)
    pos = np.zeros(T, int)
    for b in range(B):
        pos[start[b]:start[b + 1]] = lens[b] - n[b] + np.arange(n[b])
    ref = oc.rotary(x0, pos, turns_to_frequencies(steps), False)
    ref[:start[0]], ref[start[-1]:] = x0[:start[0]], x0[start[-1]:]
    assert np.all(np.abs(np64(x) - ref) <= rotary_bound(x0, ref, 32, False, 1.0, "f32"))
    assert np.array_equal(np64(x)[:start[0]], x0[:start[0]]) and np.array_equal(np64(x)[start[-1]:], x0[start[-1]:])
    assert sv.read_status(ws) == 0


def test_rotary_bad_sequences_are_left(sv):
    torch = torch_mod()
    x = torch.ones(12, 1, 64, device="cuda")
    steps, _ = sv.spec_rotary_steps(64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    # rows 0-3 good, 4-7 a length below the rows, then a decreasing start
    sv.spec_rotary(x, None, steps, q_start=i32([0, 4, 8, 6]), kv_len=i32([9, 2, 5]), workspace=ws)
    y = np64(x)
    assert np.all(y[4:] == 1) and np.any(y[:4] != 1)
    assert sv.read_status(ws) == sv.SPEC_STATUS_BAD_RANGE | sv.SPEC_STATUS_BAD_KV_LEN


def test_rotary_strides(sv):
    """q and k as views of one fused projection, outputs in another order of dimensions."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    qkv = torch.from_numpy(rng.standard_normal((37, 4 + 2 + 2, 64))).bfloat16().cuda()
    q, k = qkv[:, :4], qkv[:, 4:6]
    steps, _ = sv.spec_rotary_steps(64)
    pos = rng.integers(0, 9000, 37)
    qo = torch.empty(4, 37, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ko = torch.empty(2, 37, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    sv.spec_rotary(q, k, steps, positions=i32(pos), q_out=qo, k_out=ko)
    for x, y in ((q, qo), (k, ko)):
        ref = oc.rotary(np64(x), pos, turns_to_frequencies(steps), False)
        assert np.all(np.abs(np64(y) - ref) <= rotary_bound(np64(x), ref, 32, False, 1.0, "bf16"))


# ------------------------------------------------------------------------------ append
class Cache8:
    """A paged cache in 8 bits with garbage in every slot, and new rows with garbage around them."""

    def __init__(self, q_len, kv_len, Hkv=2, D=64, page=16, block=8, dtype="bf16", seed=0, lead=1, trail=2, layout="hnd",
                 scale=1.0):
        torch = torch_mod()
        rng = self.rng = np.random.default_rng(seed)
        self.page, self.block, self.Hkv, self.D, self.B = page, block, Hkv, D, len(q_len)
        self.start = np.cumsum([lead] + list(q_len)).astype(np.int32)
        self.kv_len = np.array(kv_len, dtype=np.int32)
        self.T = int(self.start[-1]) + trail
        per = [-(-n // page) for n in kv_len]
        self.pages = sum(per) + 2
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((self.B, max(max(per), 1)), -1, dtype=np.int32)
        for b, n in enumerate(per):
            self.table[b, :n] = order[sum(per[:b]):sum(per[:b + 1])]
        finite = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
        self.codes = [finite[rng.integers(0, 254, (self.pages, Hkv, page, D))] for _ in range(2)]
        self.exps = [rng.integers(120, 124, (self.pages, Hkv, page // block)).astype(np.uint8) for _ in range(2)]
        shape = (self.T, Hkv, D)
        self.new = [torch.from_numpy(rng.standard_normal(shape) * scale * 2.0 ** rng.integers(-3, 4, (self.T, Hkv, 1))).to(dt(dtype))
                    for _ in range(2)]
        for x in self.new:
            x[:lead] = float("nan")
            x[self.start[-1]:] = float("nan")
        self.layout = layout

    def to_device(self):
        torch = torch_mod()
        self.d_new = [x.cuda() for x in self.new]
        if self.layout == "nhd":
            both = torch.from_numpy(np.stack([c.transpose(0, 2, 1, 3) for c in self.codes], 2)).cuda()
            self.d_codes = [both[:, :, i].permute(0, 2, 1, 3).view(torch.float8_e4m3fn) for i in range(2)]
            exps = torch.from_numpy(np.stack(self.exps, 1)).cuda()
            self.d_exps = [exps[:, i] for i in range(2)]
        else:
            self.d_codes = [torch.from_numpy(c.copy()).cuda().view(torch.float8_e4m3fn) for c in self.codes]
            self.d_exps = [torch.from_numpy(e.copy()).cuda() for e in self.exps]
        self.d_table, self.d_start, self.d_len = i32(self.table), i32(self.start), i32(self.kv_len)
        return self

    def state(self):
        torch = torch_mod()
        return [x.contiguous().view(torch.uint8).cpu().numpy() for x in (*self.d_codes, *self.d_exps)]

    def append(self, sv, **kw):
        torch = torch_mod()
        ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
        sv.spec_kv8_append(*self.d_new, *self.d_codes, *self.d_exps, self.d_table, self.d_start, self.d_len, workspace=ws, **kw)
        torch.cuda.synchronize()
        return sv.read_status(ws)

    def oracle(self):
        return oc.append8(*(np64(x) for x in self.new), *self.codes, *self.exps, self.table, self.start, self.kv_len, self.block)

    def verify(self, sv):
        self.to_device()
        assert self.append(sv) == 0
        for name, got, want in zip(("k", "v", "k_exp", "v_exp"), self.state(), self.oracle()):
            assert np.array_equal(got, want), f"{name}: {np.argwhere(got != want)[:4].tolist()}"


@pytest.mark.parametrize("kw", [
    dict(q_len=[1], kv_len=[1]), dict(q_len=[1], kv_len=[8], block=8), dict(q_len=[1], kv_len=[9], block=8),
    dict(q_len=[5, 0, 3, 16], kv_len=[21, 40, 3, 17]), dict(q_len=[5, 7], kv_len=[30, 95], page=24, block=12, D=128),
    dict(q_len=[9, 2], kv_len=[50, 33], block=1), dict(q_len=[130, 1], kv_len=[200, 128], page=128, block=128, D=128),
    dict(q_len=[33] * 5, kv_len=[40, 33, 64, 47, 100], page=32, block=4, dtype="f32"),
    dict(q_len=[3] * 300, kv_len=list(range(3, 303)), page=16, block=16, Hkv=1),
    dict(q_len=[6, 5], kv_len=[60, 61], layout="nhd", D=128, Hkv=3), dict(q_len=[1000], kv_len=[1003], page=64, block=32, Hkv=8, D=128),
    dict(q_len=[20, 4], kv_len=[27, 31], scale=2.0 ** -100, dtype="f32"), dict(q_len=[20, 4], kv_len=[27, 31], scale=2.0 ** 90),
    dict(q_len=[7] * 40, kv_len=[500 + i for i in range(40)], page=3, block=3, Hkv=2), dict(q_len=[70], kv_len=[70], page=7, block=7)])
def test_append_parity(sv, kw):
    Cache8(**kw, seed=len(kw["q_len"]) + kw["kv_len"][0]).verify(sv)


def test_append_special_values(sv):
    c = Cache8([6, 6], [10, 6], D=64, block=8, dtype="f32", seed=5)
    r = int(c.start[0])
    c.new[0][r + 1, 0, 3], c.new[0][r + 2, 0, 4], c.new[0][r + 2, 0, 5] = float("nan"), float("inf"), -float("inf")
    c.new[1][r:r + 6] = 0.0                 # a block of zeros beside earlier tokens
    c.new[1][r + 6:r + 12] = 0.0            # and one on its own: the least exponent
    c.new[0][r + 6:r + 12] = float("inf")   # nothing finite
    c.new[0][r + 7, 1] = torch_mod().tensor([448.0 * 2.0 ** -3] * 63 + [-0.0])
    c.verify(sv)


def test_append_all_bf16_values(sv):
    """Every finite bf16 value of every magnitude class, rounded as the definition says."""
    torch = torch_mod()
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    v = v[torch.argsort(v.float().abs(), stable=True)][:65024].view(-1, 1, 64)
    n = v.shape[0]
    c = Cache8([n], [n], Hkv=1, D=64, page=16, block=4, lead=0, trail=0)
    c.new = [v.clone(), v.flip(0).clone()]
    c.verify(sv)


def test_append_by_single_tokens_after_rollbacks(sv):
    """Tokens one after the other, with rejected ones overwritten: the same as the definition step by step."""
    torch = torch_mod()
    c = Cache8([1], [1], Hkv=2, D=64, page=16, block=8, lead=0, trail=0, seed=9)
    c.table = np.array([[1, 0, 2]], dtype=np.int32)
    c.to_device()
    rng = np.random.default_rng(1)
    length = 0
    for step in range(14):
        n = int(rng.integers(1, 6))
        c.new = [torch.from_numpy(rng.standard_normal((n, 2, 64)) * 2.0 ** rng.integers(-4, 5)).bfloat16() for _ in range(2)]
        c.start, c.kv_len = np.array([0, n], np.int32), np.array([length + n], np.int32)
        c.d_new, c.d_start, c.d_len = [x.cuda() for x in c.new], i32(c.start), i32(c.kv_len)
        assert c.append(sv) == 0
        want = c.oracle()
        for got, ref in zip(c.state(), want):
            assert np.array_equal(got, ref), step
        c.codes, c.exps = want[:2], want[2:]
        length += int(rng.integers(1, n + 1))


def test_append_bad_data(sv):
    c = Cache8([4, 4, 4, 4], [20, 3, 40, 25], seed=3)
    c.table[2, 2] = c.pages + 7   # tokens 36 .. 39 of sequence 2
    c.table[3, 1] = -1            # tokens 21 .. 24 of sequence 3
    c.kv_len[1] = 3               # below its rows
    c.to_device()
    before = c.state()
    assert c.append(sv) == sv.SPEC_STATUS_BAD_KV_LEN | sv.SPEC_STATUS_BAD_PAGE
    good = Cache8([4, 4, 4, 4], [20, 3, 40, 25], seed=3)
    good.kv_len = np.array([20, 4, 4, 4], np.int32)
    good.start = good.start.copy()
    want = oc.append8(*(np64(x) for x in good.new), *good.codes, *good.exps, good.table, good.start[:2], good.kv_len[:1], good.block)
    for a, b, w in zip(c.state(), before, want):
        assert np.array_equal(a, w) and not np.array_equal(a, b)
    # more rows claimed than there are, by sequences that overlap, and a decreasing start: nothing outside is touched
    c.start = np.array([0, 18, 5, 18, 2], np.int32)
    c.kv_len = np.array([18, 18, 18, 18], np.int32)
    c.d_start, c.d_len = i32(c.start), i32(c.kv_len)
    assert c.append(sv) & sv.SPEC_STATUS_BAD_RANGE
    assert c.table.shape == (4, 3)


def test_append_captured_and_on_another_stream(sv):
    torch = torch_mod()
    c = Cache8([5, 3], [29, 40], D=128, Hkv=4, seed=2).to_device()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (*c.d_new, *c.d_codes, *c.d_exps, c.d_table, c.d_start, c.d_len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = c.state()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            sv.spec_kv8_append(*args, workspace=ws)
    assert all(np.array_equal(a, b) for a, b in zip(c.state(), keep))  # captured, not run
    for x in c.d_new:
        x.mul_(2)
    c.new = [x.cpu() for x in c.d_new]
    g.replay()
    torch.cuda.synchronize()
    assert sv.read_status(ws) == 0
    for got, want in zip(c.state(), c.oracle()):
        assert np.array_equal(got, want)
    d = Cache8([5, 3], [29, 40], D=128, Hkv=4, seed=2).to_device()
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_kv8_append(*d.d_new, *d.d_codes, *d.d_exps, d.d_table, d.d_start, d.d_len, stream=side)
    side.synchronize()
    for got, want in zip(d.state(), d.oracle()):
        assert np.array_equal(got, want)
