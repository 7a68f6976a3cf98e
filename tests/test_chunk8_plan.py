"""The plan of chunks over a cache in 8 bits, whose shares count what a piece costs beside its units: restated on the
host, and read back from the workspace of calls.  What a plan has to satisfy is test_chunk_plan's."""

import random

import pytest

from . import test_chunk_plan as host
from .helpers import torch_mod
from .test_chunk_plan_device import CASES, read_plan, tiles_of

EXTRA = 3


def plan(sizes, Hkv, grid, min_units, force=None, extra=EXTRA):
    """host.plan with a piece's `extra` units: shares {cta: [(tile, head, u0, u1, slot)]}, small tiles, cut tiles."""
    total, n_items = sum(sizes) * Hkv, len(sizes) * Hkv
    per = max(min_units, -(-(total + extra * n_items) // grid))
    mean = (total + host.PIECE_COST * n_items) / grid
    whole = max(max(sizes, default=0) + host.PIECE_COST, -(-n_items // grid) * mean * grid / max(n_items, 1))
    cut = mean + host.CUT_COST < 0.95 * whole if force is None else force
    big = [t for t, n in enumerate(sizes) if cut and n > per // host.FRACTION]
    among = set(big)
    small = sorted((t for t, n in enumerate(sizes) if t not in among and n > 0), key=lambda t: -sizes[t])
    items = [(t, g) for t in big for g in range(Hkv)]
    starts = [0]  # of the items on the line
    for t, _ in items:
        starts.append(starts[-1] + sizes[t] + extra)
    line = starts[-1]
    ctas = 0
    if line:
        ctas = grid if not small else min(grid, max(1, (line + per // 2) // per))
        ctas = min(ctas, -(-line // min_units))
    share = [(c + 1) * line // ctas - c * line // ctas for c in range(ctas)]
    waves = host.PIECES if ctas else 0
    for c in range(ctas):
        total, k = 0, 0
        for t, _ in items[c::ctas]:
            total += sizes[t] + extra
            if total >= line // ctas:
                break
            k += 1
        waves = min(waves, k)
    at = starts[min(waves * ctas, len(items))]
    begins = []
    for c in range(ctas):
        i = max((i for i in range(len(items)) if starts[i] <= at), default=0) if at < line else None
        begins.append(starts[i] if i is not None and at - starts[i] <= extra else at)
        lacks = share[c] - sum(sizes[items[k * ctas + c][0]] + extra for k in range(waves))
        assert lacks >= 1
        at += lacks
    assert at == line or not ctas
    begins.append(line)
    shares, cuts = {}, []
    for c in range(ctas):
        mine = [(*items[k * ctas + c], 0, sizes[items[k * ctas + c][0]], -1) for k in range(waves)]
        begin, end = begins[c], begins[c + 1]
        p = begin
        while p < end:
            i = max(i for i in range(len(items)) if starts[i] <= p)
            stop = min(end, starts[i + 1])
            is_whole = (p, stop) == (starts[i], starts[i + 1])
            u0 = 0 if p == starts[i] else p - starts[i] - extra
            mine.append((*items[i], u0, stop - starts[i] - extra, -1 if is_whole else 2 * c + (p != begin)))
            if not is_whole and p == starts[i]:
                cuts.append((*items[i], c, max(x for x in range(ctas) if begins[x] < starts[i + 1]), int(p != begin)))
            p = stop
        shares[c] = mine
    return shares, small, cuts, (ctas if ctas < grid else 0)


def check(sizes, Hkv, grid, min_units):
    for force in (None, True, False):
        for extra in (1, EXTRA):
            host.check_plan(sizes, Hkv, grid, plan(sizes, Hkv, grid, min_units, force, extra))


@pytest.mark.parametrize("seed", range(20))
def test_random_batches(seed):
    rng = random.Random(500 + seed)
    grid, Hkv = rng.choice([1, 2, 148, 152, 160]), rng.choice([1, 2, 3, 8])
    for _ in range(8):
        top = rng.choice([1, 2, 5, 40, 1000])
        sizes = [rng.randint(1, top) for _ in range(rng.choice([1, 2, 7, 60, 150]))]
        if rng.random() < 0.3:
            sizes[0] = rng.randint(1, 20000)
        check(sizes, Hkv, grid, rng.choice([1, 2, 4]))


def test_edges():
    check([], 8, 152, 2)
    check([1], 1, 152, 2)
    check([1] * 400, 8, 152, 2)
    check([248] * 32, 8, 152, 2)
    check([1000000], 1, 152, 2)
    check([1] * 639 + [3], 1, 160, 1)
    check([4] * 100, 2, 152, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [i for i, c in enumerate(CASES) if c[1] is not None])
@pytest.mark.parametrize("D", [64, 128])
def test_plan_of_a_call(case, D):
    torch = torch_mod()
    import speculative_decoding_verify_attn_gb300 as sv
    q_len, lens, Hq, Hkv, window = CASES[case]
    B, T, G, page = len(q_len), sum(q_len), Hq // Hkv, 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    start = [sum(q_len[:b]) for b in range(B + 1)]
    q = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    codes = [torch.zeros((4, Hkv, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.full((4, Hkv, 4), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.zeros((B, -(-max(lens) // page)), dtype=torch.int32, device="cuda")
    ws = torch.full((sv.spec_paged_attn8_workspace(q, codes[0], table, q, max_q=max(q_len)),), 255, dtype=torch.uint8,
                    device="cuda")
    sv.spec_paged_attn8(q, *codes, *exps, table, i32(start), i32(lens), torch.empty_like(q), max_q=max(q_len),
                        window=window, workspace=ws)
    torch.cuda.synchronize()
    short = [b for b in range(B) if q_len[b] and lens[b] < q_len[b]]
    assert sv.read_status(ws) == (sv.binding.SPEC_STATUS_BAD_KV_LEN if short else 0)
    tiles = tiles_of([0 if b in short else n for b, n in enumerate(q_len)], lens, G, window, 256, 128)
    index = {t[:2]: i for i, t in enumerate(tiles)}
    grid = min(torch.cuda.get_device_properties(0).multi_processor_count, host.MAX_GRID)
    (n_small, n_splits, ctas, first), big, small, splits = read_plan(ws, T, G, B, 256)
    assert 0 <= ctas <= grid and first == (ctas if ctas < grid else 0)
    place = lambda x: index[(x[0], x[1])]  # noqa: E731
    shares = {c: [(place(x), int(x[9]), int(x[2]) - tiles[place(x)][2], int(x[3]) - tiles[place(x)][2], int(x[4])) for x in pieces]
              for c, pieces in enumerate(big)}
    dealt = [place(x) for x in small]
    cuts = [(place(x), int(x[2]), int(x[3]), int(x[4]), int(x[5])) for x in splits]
    sizes = [t[3] for t in tiles]
    host.check_plan(sizes, Hkv, grid, (shares, dealt, cuts, first))
    want = plan(sizes, Hkv, grid, 2)
    assert shares == want[0] and sorted(dealt) == sorted(want[1]) and sorted(cuts) == sorted(want[2]) and first == want[3]
