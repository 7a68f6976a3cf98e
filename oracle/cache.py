"""Oracle of the operators around a paged KV cache in NumPy float64 and plain Python: rotary positions, the
cache in 8 bits and attention over it, pages forked and compacted, written from their definitions.  Test
infrastructure only; shares no code with the library."""

from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------------------ rotary positions
def rotary(x, positions, frequencies, pairs, amplitude=1.0, inverse=False):
    """x [T, H, D] with the first 2 * len(frequencies) values of each head turned by position * frequency."""
    x = np.array(x, dtype=np.float64)
    half = len(frequencies)
    for t, pos in enumerate(positions):
        angle = float(pos) * np.asarray(frequencies, dtype=np.longdouble)
        c, s = np.cos(angle) * amplitude, np.sin(angle) * amplitude * (-1 if inverse else 1)
        a, b = (x[t, :, 0:2 * half:2].copy(), x[t, :, 1:2 * half:2].copy()) if pairs else (
            x[t, :, :half].copy(), x[t, :, half:2 * half].copy())
        ra, rb = a * c - b * s, b * c + a * s
        if pairs:
            x[t, :, 0:2 * half:2], x[t, :, 1:2 * half:2] = ra, rb
        else:
            x[t, :, :half], x[t, :, half:2 * half] = ra, rb
    return x


def frequencies(rot, base=10000.0):
    return np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=np.longdouble)


# ------------------------------------------------------------------------------ e4m3
def _values():
    """What the 256 codes stand for."""
    v = np.zeros(256)
    for code in range(256):
        sign, e, m = -1.0 if code & 128 else 1.0, code >> 3 & 15, code & 7
        v[code] = sign * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
        if e == 15 and m == 7:
            v[code] = np.nan
    return v


VALUES = _values()
_GRID = VALUES[:127]                       # 0 .. 448
_EDGES = (_GRID[1:] + _GRID[:-1]) / 2.0    # halfway between neighbours


def encode(x):
    """Codes of the nearest values, ties to even codes, +-448 beyond it, 0x7f for NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    a = np.where(np.isnan(a), 0.0, np.minimum(a, 448.0))
    code = np.searchsorted(_EDGES, a, side="left")     # ties: the lower code
    tie = (code < 126) & (a == _EDGES[np.minimum(code, 125)])
    code = np.where(tie & (code & 1 == 1), code + 1, code)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def needed(amax):
    """The least exponent in [-64, 64] whose scale brings amax within 448."""
    e = -64
    while e < 64 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def clamped(byte):
    return min(max(int(byte), 63), 191) - 127


def append8(k_new, v_new, k_pages, v_pages, k_exp, v_exp, table, q_start, kv_len, block):
    """The codes [pages, Hkv, page_size, D] and exponent bytes [pages, Hkv, blocks] after the append."""
    out = [x.copy() for x in (k_pages, v_pages, k_exp, v_exp)]
    size = k_pages.shape[2]
    for b in range(len(kv_len)):
        r0, n, end = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        first = end - n
        for t0 in range(first // block * block, end, block):
            lo, hi = max(t0, first), min(t0 + block, end)
            if hi <= lo:
                continue
            page, at = int(table[b, t0 // size]), t0 % size
            for new, codes, exp in ((k_new, out[0], out[2]), (v_new, out[1], out[3])):
                for g in range(codes.shape[1]):
                    x = np.asarray(new[r0 + lo - first:r0 + hi - first, g], dtype=np.float64)
                    fin = np.abs(x[np.isfinite(x)])
                    e = needed(fin.max(initial=0.0))
                    if lo > t0:
                        old = clamped(exp[page, g, at // block])
                        e = max(e, old)
                        if e > old:
                            was = VALUES[codes[page, g, at:at + lo - t0]] * 2.0 ** (old - e)
                            codes[page, g, at:at + lo - t0] = encode(was)
                    exp[page, g, at // block] = e + 127
                    codes[page, g, at + lo - t0:at + hi - t0] = encode(x * 2.0 ** -e)
    return out


def stands_for(codes, exp):
    """The values of a cache: codes [..., page_size, D], exponent bytes [..., blocks]."""
    block = codes.shape[-2] // exp.shape[-1]
    e = np.repeat(np.clip(exp.astype(np.int64), 63, 191) - 127, block, axis=-1)
    return VALUES[codes] * 2.0 ** e[..., None].astype(np.float64)


def paged_attn8(q, codes, exps, table, q_start, kv_len, window=0, scale=0.0):
    """o [T, Hq, D], with what the error bound is made of, per row and head: A = sum p |v|, W = (the largest p 2^ev) *
    sum |v / 2^ev|, and the same with 2^ev replaced by the largest scale among 32 neighbouring keys, together; and the
    largest scale * sum |q k|."""
    T, Hq, D = q.shape
    scale = scale or D ** -0.5
    size, Hkv = codes[0].shape[2], codes[0].shape[1]
    block = size // exps[0].shape[2]
    o, A, W, S = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape), 0.0
    for b in range(len(kv_len)):
        r0, r1, length = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        n = r1 - r0
        if n == 0:
            continue
        low = max(0, length - n + 1 - window) if window > 0 else 0
        t = np.arange(low, length)
        page, slot = table[b, t // size], t % size
        for g in range(Hkv):
            ke, ve = (np.clip(x[page, g, slot // block].astype(np.int64), 63, 191) - 127.0 for x in exps)
            k, v8 = VALUES[codes[0][page, g, slot]] * 2.0 ** ke[:, None], VALUES[codes[1][page, g, slot]]
            v = v8 * 2.0 ** ve[:, None]
            top = np.array([ve[t // 32 == i // 32].max() for i in t])  # of the keys that the chunk sees
            near = np.abs(v8) * 2.0 ** (ve - top)[:, None]
            for j in range(n):
                pos = length - n + j
                seen = (t <= pos) & ((t > pos - window) if window > 0 else True)
                for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                    s = k[seen] @ q[r0 + j, h] * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o[r0 + j, h], A[r0 + j, h] = p @ v[seen], p @ np.abs(v[seen])
                    W[r0 + j, h] = (p * 2.0 ** ve[seen]).max() * np.abs(v8[seen]).sum(0) + \
                        (p * 2.0 ** top[seen]).max() * near[seen].sum(0)
                    S = max(S, float((np.abs(k[seen]) @ np.abs(q[r0 + j, h])).max()) * abs(scale))
    return o, A, W, S


# ------------------------------------------------------------------------------ pages
def page_fork(table, held, kv_len, refs, parent, grow, page_size):
    """(table, held, kv_len, refs, copies [(from, to)]) after one step, or None if the free pages do not suffice.
    Rows and pages are looked at one after the other."""
    B = len(parent)
    pages = lambda n: -(-n // page_size)  # noqa: E731
    refs = [int(x) for x in refs]
    rows, before = [], []
    for b in range(B):
        n = int(kv_len[parent[b]]) if parent[b] >= 0 else 0
        before.append(n)
        rows.append([int(x) for x in table[parent[b], :pages(n)]] if parent[b] >= 0 else [])
    for b in range(B):
        for e in table[b, :held[b]]:
            refs[e] -= 1
        for e in rows[b]:
            refs[e] += 1
    grown = [int(grow[b]) if parent[b] >= 0 else 0 for b in range(B)]
    writers = {}
    for b in range(B):
        if grown[b] > 0 and before[b] % page_size:
            writers.setdefault(rows[b][-1], []).append(b)
    copier = []
    for b in range(B):
        last = rows[b][-1] if grown[b] > 0 and before[b] % page_size else None
        copier.append(last is not None and refs[last] > 1 and not (len(writers[last]) == refs[last] and writers[last][0] == b))
    free = [i for i, n in enumerate(refs) if n <= 0]
    copies, after = [], list(refs)
    for b in range(B):
        need = pages(before[b] + grown[b])
        if len(free) < copier[b] + need - len(rows[b]):
            return None
        if copier[b]:
            to = free.pop(0)
            copies.append((rows[b][-1], to))
            after[rows[b][-1]] -= 1
            after[to] = 1
            rows[b][-1] = to
        while len(rows[b]) < need:
            to = free.pop(0)
            after[to] = 1
            rows[b].append(to)
    out = np.array(table)
    for b in range(B):
        out[b, :len(rows[b])] = rows[b]
    return (out, np.array([len(r) for r in rows], np.int32), np.array([n + g for n, g in zip(before, grown)], np.int32),
            np.array(after, np.int32), copies)


def page_compact(table, held, refs):
    """(table, refs, moved, live, copies) of a pool."""
    n = len(refs)
    used = [i for i in range(n) if refs[i] > 0]
    live = len(used)
    gaps = [i for i in range(live) if refs[i] <= 0]
    copies = list(zip([i for i in used if i >= live], gaps))
    moved = np.array([i if refs[i] > 0 else -1 for i in range(n)], np.int32)
    after = np.array([max(int(x), 0) if i < live else 0 for i, x in enumerate(refs)], np.int32)
    for a, b in copies:
        moved[a], after[b] = b, refs[a]
    out = np.array(table)
    for b in range(len(held)):
        out[b, :held[b]] = moved[table[b, :held[b]]]
    return out, after, moved, live, copies
