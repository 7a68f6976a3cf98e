"""The chunk kernels' plan, restated on the host: every (tile, kv head, unit) is computed exactly once, a share
never holds more pieces than its list has room for, records and cut tiles stay within their arrays, and a
cut tile's records are the ones its merge reads.  (The device code is chunk_plan.cu.)"""

import random

import pytest

MAX_GRID, FRACTION, PIECES = 160, 4, 8
PIECE_COST, CUT_COST = 3, 7


def plan(sizes, Hkv, grid, min_units, force=None):
    """(force: cut or not, whatever the estimate says.)  Shares {cta: [(tile, head, u0, u1, slot)]}, small tiles in dealing order, cut tiles."""
    total = sum(sizes)
    per = max(min_units, -(-total * Hkv // grid))
    items = len(sizes) * Hkv
    mean = (total * Hkv + PIECE_COST * items) / grid
    whole = max(max(sizes, default=0) + PIECE_COST, -(-items // grid) * mean * grid / max(items, 1))
    cut = mean + CUT_COST < 0.95 * whole if force is None else force
    big = [t for t, n in enumerate(sizes) if cut and n > per // FRACTION]
    small = sorted((t for t, n in enumerate(sizes) if t not in set(big) and n > 0), key=lambda t: -sizes[t])
    at = [0]
    for t in big:
        at.append(at[-1] + sizes[t])
    line = at[-1] * Hkv
    ctas = 0
    if line:
        ctas = grid if not small else min(grid, max(1, (line + per // 2) // per))
        ctas = min(ctas, -(-line // min_units))
    share = -(-line // ctas) if ctas else 1
    items = [(t, g) for t in big for g in range(Hkv)]
    waves = PIECES if ctas else 0
    for c in range(ctas):
        total, k = 0, 0
        for t, _ in items[c::ctas]:
            total += sizes[t]
            if total >= share:
                break
            k += 1
        waves = min(waves, k)
    first = waves * ctas
    rest = line if first >= len(items) else line - sum(sizes[t] for t, _ in items[first:])
    shares, cuts, starts = {}, [], []
    p = rest
    for c in range(ctas):
        starts.append(p)
        p += share - sum(sizes[items[k * ctas + c][0]] for k in range(waves))
    starts.append(p)
    assert all(a < b for a, b in zip(starts, starts[1:]))  # every share lacks at least a unit
    for c in range(ctas):
        mine = [(*items[k * ctas + c], 0, sizes[items[k * ctas + c][0]], -1) for k in range(waves)]
        begin, end = starts[c], min(line, starts[c + 1])
        p = begin
        while p < end:
            j = max(i for i in range(len(big)) if at[i] * Hkv <= p)
            n = sizes[big[j]]
            g = (p - at[j] * Hkv) // n
            start = at[j] * Hkv + g * n
            stop = min(end, start + n)
            whole = p == start and stop == start + n
            mine.append((big[j], g, p - start, stop - start, -1 if whole else 2 * c + (0 if p == begin else 1)))
            if not whole and p == start:
                last = max(x for x in range(ctas) if starts[x] <= start + n - 1)
                cuts.append((big[j], g, c, last, 0 if p == begin else 1))
            p = stop
        shares[c] = mine
    return shares, small, cuts, (ctas if ctas < grid else 0)


def check(sizes, Hkv, grid, min_units):
    for force in (None, True, False):
        check_plan(sizes, Hkv, grid, plan(sizes, Hkv, grid, min_units, force))


def check_plan(sizes, Hkv, grid, made):
    shares, small, cuts, first = made
    assert sum(n > 0 for n in sizes) >= len(cuts) / Hkv and len(cuts) <= MAX_GRID
    seen, slots = {}, {}
    for c, mine in shares.items():
        assert len(mine) <= PIECES
        for tile, g, u0, u1, slot in mine:
            assert 0 <= u0 < u1 <= sizes[tile]
            seen.setdefault((tile, g), []).append((u0, u1))
            if slot >= 0:
                assert slot < 2 * MAX_GRID and slot not in slots
                slots[slot] = (tile, g, u0)
    ctas = grid - first
    dealt = [c for c in range(grid) if c >= first]
    for k in range(-(-len(small) * Hkv // ctas)):
        for at, c in enumerate(dealt):
            idx = k * ctas + (ctas - 1 - at if k & 1 else at)
            if idx < len(small) * Hkv:
                seen.setdefault((small[idx // Hkv], idx % Hkv), []).append((0, sizes[small[idx // Hkv]]))
    for tile, n in enumerate(sizes):
        for g in range(Hkv if n else 0):
            pieces = sorted(seen.pop((tile, g)))
            assert pieces[0][0] == 0 and pieces[-1][1] == n
            assert all(a[1] == b[0] for a, b in zip(pieces, pieces[1:]))
    assert not seen
    # a merge reads every record of its tile, in key order
    for tile, g, c0, c1, f in cuts:
        recs = [2 * c0 + (f if i == 0 else 2 * i) for i in range(c1 - c0 + 1)]
        got = [slots.pop(r) for r in recs]
        assert all(x[:2] == (tile, g) for x in got) and [x[2] for x in got] == sorted(x[2] for x in got)
    assert not slots


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    rng = random.Random(seed)
    grid, Hkv = rng.choice([1, 2, 148, 152, 160]), rng.choice([1, 2, 3, 8, 32])
    for _ in range(25):
        top = rng.choice([1, 2, 5, 40, 1000])
        sizes = [rng.randint(1, top) for _ in range(rng.choice([1, 2, 7, 60, 300]))]
        if rng.random() < 0.3:
            sizes[0] = rng.randint(1, 20000)
        check(sizes, Hkv, grid, rng.choice([1, 2, 4]))


def test_edges():
    check([], 8, 152, 2)
    check([1], 1, 152, 2)
    check([1] * 5000, 8, 152, 2)
    check([248] * 32, 8, 152, 2)
    check([1000000], 1, 152, 2)
    check([1] * 639 + [3], 1, 160, 1)
