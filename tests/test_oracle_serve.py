"""Pins of the serving operators' oracle: closed forms, the dense verify oracle, and scipy."""

import numpy as np
import pytest
from scipy.special import log_softmax, softmax

from oracle import attn as oa
from oracle import serve as os_


def paged_inputs(rng, q_len, kv_len, Hq, Hkv, D, page):
    T = sum(q_len)
    per = [-(-n // page) for n in kv_len]
    pages = sum(per) + 2
    order = rng.permutation(pages)
    table = np.full((len(q_len), max(per)), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    return (rng.standard_normal((T, Hq, D)), rng.standard_normal((pages, Hkv, page, D)),
            rng.standard_normal((pages, Hkv, page, D)), table, start, np.array(kv_len, dtype=np.int32))


def test_paged_equals_dense_verify():
    rng = np.random.default_rng(1)
    q, kp, vp, table, start, kv = paged_inputs(rng, [3, 3], [17, 29], 4, 2, 8, 5)
    Lmax = 30
    k = np.zeros((2, 2, Lmax, 8))
    v = np.zeros_like(k)
    for b in range(2):
        for t in range(kv[b]):
            k[b, :, t], v[b, :, t] = kp[table[b, t // 5], :, t % 5], vp[table[b, t // 5], :, t % 5]
    ref = oa.verify_attn(q.reshape(2, 3, 4, 8), k, v, kv)
    o, _, _ = os_.paged_attn(q, kp, vp, table, start, kv)
    assert np.max(np.abs(o - ref.reshape(6, 4, 8))) < 1e-12


def test_window_is_the_last_tokens():
    rng = np.random.default_rng(2)
    q, kp, vp, table, start, kv = paged_inputs(rng, [4, 0, 1], [11, 3, 9], 2, 1, 4, 4)
    vp[:] = 0
    # v holds the token's index: a window of one reads the row's own position
    for b in range(3):
        for t in range(kv[b]):
            vp[table[b, t // 4], :, t % 4] = t
    o, _, _ = os_.paged_attn(q, kp, vp, table, start, kv, window=1)
    assert np.allclose(o[:4, 0, 0], [7, 8, 9, 10]) and np.allclose(o[4], 8)
    wide, _, _ = os_.paged_attn(q, kp, vp, table, start, kv, window=11)
    full, _, _ = os_.paged_attn(q, kp, vp, table, start, kv)
    assert np.allclose(wide, full)


def test_prefill_equals_masked_softmax():
    rng = np.random.default_rng(3)
    start = np.array([0, 5, 5, 12])
    q, k, v = (rng.standard_normal((12, h, 6)) for h in (4, 2, 2))
    seq = np.repeat([0, 2], [5, 7])
    i, j = np.arange(12)[:, None], np.arange(12)[None]
    for window in (0, 3):
        seen = (seq[:, None] == seq[None]) & (j <= i) & ((i - j < window) | (window == 0))
        o, _, _ = os_.prefill_attn(q, k, v, start, window)
        for h in range(4):
            s = np.where(seen, q[:, h] @ k[:, h // 2].T * 6 ** -0.5, -np.inf)
            assert np.max(np.abs(o[:, h] - softmax(s, axis=1) @ v[:, h // 2])) < 1e-12


def test_append_places_rows():
    rng = np.random.default_rng(4)
    q, kp, vp, table, start, kv = paged_inputs(rng, [2, 3], [9, 4], 2, 2, 4, 4)
    kn, vn = rng.standard_normal((5, 2, 4)), rng.standard_normal((5, 2, 4))
    k2, v2 = os_.append_pages(kp, vp, table, start, kv, kn, vn)
    assert np.array_equal(k2[table[0, 1], :, 3], kn[0]) and np.array_equal(k2[table[0, 2], :, 0], kn[1])
    assert np.array_equal(v2[table[1, 0], :, 1:4].transpose(1, 0, 2), vn[2:])
    assert (k2 != kp).any(axis=(1, 3)).sum() == 5


def test_logprobs_against_scipy_and_ties():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 50)) * 3
    x[1, 10:] = -np.inf
    x[2, :] = np.round(x[2])
    x[3, :] = -np.inf
    tok = np.array([3, 20, -1, 7])
    lp, ent, ids, top = os_.token_logprobs(x, tok, 12)
    ref = log_softmax(x[:3], axis=1)
    assert np.isclose(lp[0], ref[0, 3]) and lp[1] == -np.inf and lp[2] == 0 and lp[3] == -np.inf
    with np.errstate(invalid="ignore"):
        H = -np.nansum(np.exp(ref) * ref, axis=1)
    assert np.allclose(ent[:3], H) and ent[3] == 0
    for r in range(3):
        pairs = sorted(((-x[r, v], v) for v in range(50)))[:12]
        assert [v for _, v in pairs] == list(ids[r])
        assert np.array_equal(top[r], ref[r, ids[r]]) or np.allclose(top[r][np.isfinite(top[r])],
                                                                    ref[r, ids[r]][np.isfinite(top[r])])
    assert list(ids[3]) == list(range(12)) and np.all(top[3] == -np.inf)
