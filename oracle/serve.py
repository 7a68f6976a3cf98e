"""Oracle of the serving operators in NumPy float64: chunk attention over a paged cache, packed prompt
attention and token log probabilities, written from their definitions (one row at a time).  Test
infrastructure only; shares no code with the library."""

from __future__ import annotations

import numpy as np


def _attend_row(q, keys, values, scale):
    """softmax(scale * keys @ q) @ values, the sum of p|v|, and the largest scale * sum |q k|."""
    s = keys @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ values, p @ np.abs(values), float(np.max(np.abs(keys) @ np.abs(q))) * abs(scale)


def _attend_chunk(q, k, v, n, length, window, scale):
    """q [n, Hq, D]; k, v [Hkv, length, D] -> (o, sum p|v|) [n, Hq, D], largest sum of |q k|."""
    Hq, Hkv = q.shape[1], k.shape[0]
    o, a, big = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for j in range(n):
        pos = length - n + j
        lo = max(0, pos + 1 - window) if window > 0 else 0
        for h in range(Hq):
            g = h // (Hq // Hkv)
            o[j, h], a[j, h], b = _attend_row(q[j, h], k[g, lo:pos + 1], v[g, lo:pos + 1], scale)
            big = max(big, b)
    return o, a, big


def append_pages(k_pages, v_pages, page_table, q_start, kv_len, k_new, v_new):
    """The caches [pages, Hkv, page_size, D] after the append of every sequence's new rows."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    size = k_pages.shape[2]
    for b in range(len(kv_len)):
        n = int(q_start[b + 1] - q_start[b])
        for j in range(n):
            t = int(kv_len[b]) - n + j
            page = int(page_table[b, t // size])
            k_pages[page, :, t % size] = k_new[q_start[b] + j]
            v_pages[page, :, t % size] = v_new[q_start[b] + j]
    return k_pages, v_pages


def paged_attn(q, k_pages, v_pages, page_table, q_start, kv_len, window=0, scale=0.0):
    """Rows of every sequence's chunk over its pages: o [T, Hq, D] (zeros in rows of no sequence), the
    bound's sum of p|v|, and the largest scale * sum |q k|."""
    T, Hq, D = q.shape
    scale = scale or D ** -0.5
    size = k_pages.shape[2]
    o, a, big = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for b in range(len(kv_len)):
        r0, r1, length = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if r1 == r0:
            continue
        lo = max(0, length - (r1 - r0) + 1 - window) if window > 0 else 0
        k = np.zeros((k_pages.shape[1], length, D))
        v = np.zeros_like(k)
        for t in range(lo, length):  # tokens before every row's window are not looked up
            page = int(page_table[b, t // size])
            k[:, t], v[:, t] = k_pages[page, :, t % size], v_pages[page, :, t % size]
        o[r0:r1], a[r0:r1], x = _attend_chunk(q[r0:r1], k, v, r1 - r0, length, window, scale)
        big = max(big, x)
    return o, a, big


def prefill_attn(q, k, v, seq_start, window=0, scale=0.0):
    """Packed prompts, each causal within itself; outputs as paged_attn's."""
    D = q.shape[2]
    scale = scale or D ** -0.5
    o, a, big = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for r0, r1 in zip(seq_start[:-1], seq_start[1:]):
        if r1 > r0:
            o[r0:r1], a[r0:r1], x = _attend_chunk(q[r0:r1], k[r0:r1].transpose(1, 0, 2), v[r0:r1].transpose(1, 0, 2),
                                                  r1 - r0, r1 - r0, window, scale)
            big = max(big, x)
    return o, a, big


def token_logprobs(logits, tokens, K=0):
    """logprobs [N] (0 for ids outside the row), entropy [N], top ids and their log probabilities
    [N, K], and sum p |log p| per row for the error bound."""
    N, V = logits.shape
    lp, ent = np.zeros(N), np.zeros(N)
    ids, top = np.zeros((N, K), dtype=np.int32), np.zeros((N, K))
    for r in range(N):
        x = logits[r].astype(np.float64)
        m = x.max()
        if m == -np.inf:
            logp = np.full(V, -np.inf)
        else:
            logp = x - m - np.log(np.exp(x - m).sum())
            p = np.exp(logp)
            ent[r] = -(p[p > 0] * logp[p > 0]).sum()
        if 0 <= tokens[r] < V:
            lp[r] = logp[tokens[r]]
        order = sorted(range(V), key=lambda i: (-x[i], i))[:K] if V <= 4096 else \
            np.lexsort((np.arange(V), -x))[:K]
        ids[r] = order
        top[r] = logp[order]
    return lp, ent, ids, top
