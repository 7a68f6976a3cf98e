"""Pins of the cache operators' oracle: closed forms, brute force and hand-worked cases."""

import math

import numpy as np
import pytest

from oracle import cache as oc
from oracle import serve as os_


def test_rotary_is_a_complex_product_and_has_an_inverse():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 10))
    f = oc.frequencies(8, 100.0)
    pos = [0, 7, -5]
    for pairs in (False, True):
        y = oc.rotary(x, pos, f, pairs, amplitude=1.5)
        assert np.allclose(y[0, :, :8], 1.5 * x[0, :, :8]) and np.array_equal(y[..., 8:], x[..., 8:])
        a = x[1, 0, 0:8:2] + 1j * x[1, 0, 1:8:2] if pairs else x[1, 0, :4] + 1j * x[1, 0, 4:8]
        z = 1.5 * a * np.exp(1j * 7 * f.astype(float))
        got = y[1, 0, 0:8:2] + 1j * y[1, 0, 1:8:2] if pairs else y[1, 0, :4] + 1j * y[1, 0, 4:8]
        assert np.allclose(got, z)
        assert np.allclose(oc.rotary(oc.rotary(x, pos, f, pairs), pos, f, pairs, inverse=True), x)


def test_rotary_scores_depend_on_distance_only():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 8))
    f = oc.frequencies(8)
    s = [float((oc.rotary(q, [p + 3], f, True) * oc.rotary(k, [p], f, True)).sum()) for p in (0, 11, 1000)]
    assert np.allclose(s, s[0])


def test_e4m3_values_and_rounding():
    v = oc.VALUES
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448 and np.isnan(v[0x7F])
    fin = np.array([c for c in range(256) if c & 127 != 127])
    assert np.array_equal(oc.encode(v[fin]), fin)
    assert oc.encode([17.0, 19.0, 500.0, -1e9, np.nan, 2.0 ** -10, 3 * 2.0 ** -10]).tolist() == [
        oc.encode(16.0), oc.encode(20.0), 0x7E, 0xFE, 0x7F, 0, 2]
    rng = np.random.default_rng(3)
    x = rng.standard_normal(500) * 2.0 ** rng.integers(-11, 10, 500)
    best = [np.abs(v[fin] - np.clip(t, -448, 448)).min() for t in x]
    assert np.array_equal(np.abs(v[oc.encode(x)] - np.clip(x, -448, 448)), best)


def test_needed_exponent():
    for a in (1e-30, 0.4, 448.0, 448.0000001, 449.0, 896.0, 1e10):
        e = oc.needed(a)
        assert a <= 448 * 2.0 ** e and (e == -64 or a > 448 * 2.0 ** (e - 1))
    assert oc.needed(0.0) == -64 and oc.needed(1e38) == 64


def test_append_keeps_values_when_a_block_grows():
    """One token at a time, the last far larger: earlier values stay, exactly, where they do not become subnormal."""
    D, block = 64, 4
    rng = np.random.default_rng(4)
    x = rng.choice([1.0, -2.0, 3.0, 0.5], (4, 1, D))
    x[3] *= 64
    codes = [np.full((2, 1, 8, D), 0x55, np.uint8) for _ in range(2)]
    exp = [np.full((2, 1, 2), 200, np.uint8) for _ in range(2)]
    table = np.array([[1]])
    for t in range(4):
        codes[0], codes[1], exp[0], exp[1] = oc.append8(x[t:t + 1], -x[t:t + 1], *codes, *exp, table, [0, 1], [t + 1], block)
    assert np.array_equal(oc.stands_for(codes[0], exp[0])[1, 0, :4], x[:, 0])
    assert np.array_equal(oc.stands_for(codes[1], exp[1])[1, 0, :4], -x[:, 0])
    assert np.all(codes[0][0] == 0x55) and np.all(codes[0][1, :, 4:] == 0x55) and exp[0][1, 0, 1] == 200


def test_attention_is_that_of_the_values():
    rng = np.random.default_rng(5)
    codes = [rng.integers(0, 120, (5, 2, 8, 64)).astype(np.uint8) for _ in range(2)]
    exps = [rng.integers(118, 124, (5, 2, 4)).astype(np.uint8) for _ in range(2)]
    q = rng.standard_normal((6, 4, 64)) * 0.01
    table, start, lens = np.array([[4, 1, 0], [2, 3, 0]]), [0, 5, 6], [13, 11]
    for window in (0, 7):
        o, A, W, S = oc.paged_attn8(q, codes, exps, table, start, lens, window)
        ref, A2, S2 = os_.paged_attn(q, *(oc.stands_for(c, e) for c, e in zip(codes, exps)), table, start, lens, window)
        assert np.allclose(o, ref, rtol=1e-12) and np.allclose(A, A2) and np.isclose(S, S2) and np.all(W >= A * 0.99)


def test_fork_by_hand():
    # two rows of 6 tokens on pages of 4, sharing page 3; row 1 takes over row 0, both write two tokens
    table = np.array([[3, 5, 0], [3, 1, 0]])
    t, held, lens, refs, copies = oc.page_fork(table, [2, 2], [6, 6], [0, 1, 0, 2, 0, 1], [0, 0], [2, 3], 4)
    # page 1 is given back; pages 3 and 5 have two holders; both rows write to page 5: row 0 keeps it
    assert t.tolist() == [[3, 5, 0], [3, 0, 1]] and copies == [(5, 0)]
    assert held.tolist() == [2, 3] and lens.tolist() == [8, 9] and refs.tolist() == [1, 1, 0, 2, 0, 1]
    assert oc.page_fork(table, [2, 2], [6, 6], [1, 1, 1, 2, 1, 1], [0, 0], [2, 3], 4) is None


def test_compact_by_hand():
    t, refs, moved, live, copies = oc.page_compact(np.array([[6, 1, 9], [4, 9, 9]]), [2, 1], [0, 2, 0, 0, 1, 0, 3])
    assert live == 3 and copies == [(4, 0), (6, 2)] and moved.tolist() == [-1, 1, -1, -1, 0, -1, 2]
    assert t.tolist() == [[2, 1, 9], [0, 9, 9]] and refs.tolist() == [1, 2, 3, 0, 0, 0, 0]


@pytest.mark.parametrize("kind", range(5))
def test_rotary_steps_of_the_library(kind):
    """The host's table against the formulas (the library is built, no GPU is used)."""
    from speculative_decoding_verify_attn_gb300 import build
    import speculative_decoding_verify_attn_gb300 as sv
    build.build()
    rot, base, factor, length, low, high = 64, 10000.0, 8.0, 4096.0, 1.0, 32.0
    if kind == sv.SPEC_ROTARY_BANDS:
        high = 4.0
    steps, amp = sv.spec_rotary_steps(rot, base, kind=kind, factor=factor, length=length, low=low, high=high, device="cpu")
    want = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        wave = 2 * math.pi / f
        if kind == sv.SPEC_ROTARY_LINEAR:
            f /= factor
        elif kind == sv.SPEC_ROTARY_NTK:
            f = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == sv.SPEC_ROTARY_BANDS:
            if wave > length / low:
                f /= factor
            elif wave >= length / high:
                share = (length / wave - low) / (high - low)
                f = share * f + (1 - share) * f / factor
        elif kind == sv.SPEC_ROTARY_YARN:
            at = lambda turns: rot * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
            a, b = math.floor(at(high)), math.ceil(at(low))
            r = min(max((i - a) / (b - a), 0), 1)
            f = f * (1 - r) + f / factor * r
        want.append(f)
    got = steps.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    assert np.allclose(got, want, rtol=1e-13, atol=0)
    assert np.isclose(amp, 1 + 0.1 * math.log(factor) if kind == sv.SPEC_ROTARY_YARN else 1.0)


def test_rotary_steps_refusals():
    from speculative_decoding_verify_attn_gb300 import build
    import speculative_decoding_verify_attn_gb300 as sv
    build.build()
    for kw in (dict(rot=7), dict(rot=0), dict(rot=-2), dict(rot=2048), dict(base=1.0), dict(base=float("inf")), dict(kind=5),
               dict(kind=1, factor=0.5), dict(kind=2, factor=float("nan")), dict(kind=2, rot=2), dict(kind=3, length=0.0),
               dict(kind=4, length=100.0, low=32.0, high=1.0)):
        with pytest.raises(sv.SpecError):
            sv.spec_rotary_steps(**{**dict(rot=64, factor=2.0, length=4096.0, device="cpu"), **kw})
