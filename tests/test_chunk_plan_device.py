"""The chunk kernels' plan as the device makes it: read back from the workspace after a call and held against
what every plan has to satisfy (each unit of each tile computed once, at most eight pieces of cut tiles a CTA,
records that no two pieces share and that the merge of their tile reads).  And the host's restatement with the
costs of the fp32 kernel."""

import random

import numpy as np
import pytest

from . import test_chunk_plan as host
from .helpers import torch_mod

MAX_GRID, PIECES = host.MAX_GRID, host.PIECES


@pytest.mark.parametrize("seed", range(10))
def test_host_restatement_with_fp32_costs(seed, monkeypatch):
    monkeypatch.setattr(host, "PIECE_COST", 1)
    monkeypatch.setattr(host, "CUT_COST", 3)
    rng = random.Random(1000 + seed)
    for _ in range(25):
        top = rng.choice([1, 2, 5, 40, 1000])
        sizes = [rng.randint(1, top) for _ in range(rng.choice([1, 2, 7, 60, 300]))]
        host.check(sizes, rng.choice([1, 2, 3, 8]), rng.choice([1, 148, 152]), 2)


def tiles_of(q_len, kv_len, G, window, row_tile, unit):
    """(sequence, first row, first unit, units) of every row tile, from the definition."""
    out = []
    for b, (n, length) in enumerate(zip(q_len, kv_len)):
        for row0 in range(0, n * G, row_tile):
            first, last = row0 // G, (min(n * G, row0 + row_tile) - 1) // G
            base = length - n
            lo = max(0, base + first + 1 - window) if window else 0
            u0, u1 = lo // unit, (base + last) // unit + 1
            out.append((b, row0, u0, u1 - u0))
    return out


def up256(n):
    return (n + 255) & ~255


def read_plan(ws, T, G, B, row_tile):
    """Header, pieces per CTA, small tiles, cut tiles of a workspace (ChunkPlan, ChunkItem, ChunkSplit)."""
    raw = ws.cpu().numpy()
    ints = lambda at, n: raw[at:at + 4 * n].view(np.int32)  # noqa: E731
    at = [256, 512]
    at.append(up256(at[1] + MAX_GRID * 4))
    at.append(up256(at[2] + MAX_GRID * PIECES * 48))
    at.append(up256(at[3] + (T * G // row_tile + B) * 48))
    n_small, n_splits, ctas, first = (int(x) for x in ints(at[0], 4))
    count = ints(at[1], MAX_GRID)
    big = ints(at[2], MAX_GRID * PIECES * 12).reshape(MAX_GRID, PIECES, 12)
    return (n_small, n_splits, ctas, first), [big[c, :count[c]] for c in range(ctas)], \
        ints(at[3], n_small * 12).reshape(-1, 12), ints(at[4], n_splits * 8).reshape(-1, 8)


CASES = [  # q_len, kv_len (None: prompts), Hq, Hkv, window
    ([2048], [9000], 8, 2, 0),
    ([300, 1, 0, 64, 700], [5000, 20000, 3, 64, 701], 8, 2, 0),
    ([70] * 80, list(range(100, 8100, 100)), 4, 1, 0),
    ([64] + [64] * 450, [16384] + [64] * 450, 8, 2, 0),
    ([500, 1500, 40, 1200], None, 8, 2, 0),
    ([1, 3000], None, 2, 2, 0),
    ([60] * 100, None, 12, 4, 0),
    ([900, 2000, 5], [4000, 9000, 30000], 8, 2, 1500),
    ([1500, 2500], None, 6, 2, 1200),
    ([40], [100000], 4, 1, 0),
    ([33] * 7, [60000, 10, 0, 70, 50000, 33, 40], 1, 1, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_plan_of_a_call(case, dtype):
    torch = torch_mod()
    import speculative_decoding_verify_attn_gb300 as sv
    q_len, kv_len, Hq, Hkv, window = CASES[case]
    t, row_tile, unit = (torch.bfloat16, 256, 128) if dtype == "bf16" else (torch.float32, 64, 64)
    B, T, G, page = len(q_len), sum(q_len), Hq // Hkv, 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    start = [sum(q_len[:b]) for b in range(B + 1)]
    q = torch.zeros((T, Hq, 64), dtype=t, device="cuda")
    if kv_len is None:
        lens = list(q_len)
        k = torch.zeros((T, Hkv, 64), dtype=t, device="cuda")
        ws = torch.full((sv.spec_prefill_attn_workspace(q, k, i32(start), q),), 255, dtype=torch.uint8, device="cuda")
        sv.spec_prefill_attn(q, k, k, i32(start), torch.empty_like(q), window=window, workspace=ws)
    else:
        lens = list(kv_len)
        k = torch.zeros((4, Hkv, page, 64), dtype=t, device="cuda")
        table = torch.zeros((B, -(-max(lens) // page)), dtype=torch.int32, device="cuda")
        ws = torch.full((sv.spec_paged_attn_workspace(q, k, table, q, max_q=max(q_len)),), 255, dtype=torch.uint8,
                        device="cuda")
        sv.spec_paged_attn(q, k, k.clone(), table, i32(start), i32(lens), torch.empty_like(q), max_q=max(q_len),
                           window=window, workspace=ws)
    torch.cuda.synchronize()
    short = [b for b in range(B) if q_len[b] and lens[b] < q_len[b]]
    assert sv.read_status(ws) == (sv.binding.SPEC_STATUS_BAD_KV_LEN if short else 0)
    # sequences without keys have no tiles
    tiles = tiles_of([0 if b in short else n for b, n in enumerate(q_len)], lens, G, window, row_tile, unit)
    index = {t[:2]: i for i, t in enumerate(tiles)}
    grid = min(torch.cuda.get_device_properties(0).multi_processor_count, MAX_GRID)
    (n_small, n_splits, ctas, first), big, small, splits = read_plan(ws, T, G, B, row_tile)
    assert 0 <= ctas <= grid and first == (ctas if ctas < grid else 0)

    def own_numbers(x, tile):
        b, row0, u0, n = tile
        lo = max(0, lens[b] - q_len[b] + 1 - window) if window else 0
        assert (x[5], x[6], x[7], x[8]) == (start[b], q_len[b], lens[b], lo)

    shares, dealt, cuts = {}, [], []
    for c, pieces in enumerate(big):
        assert len(pieces) <= PIECES
        shares[c] = []
        for x in pieces:
            i = index[(x[0], x[1])]
            own_numbers(x, tiles[i])
            shares[c].append((i, int(x[9]), int(x[2]) - tiles[i][2], int(x[3]) - tiles[i][2], int(x[4])))
    for x in small:
        i = index[(x[0], x[1])]
        own_numbers(x, tiles[i])
        assert x[4] == -1 and (x[2], x[3]) == (tiles[i][2], tiles[i][2] + tiles[i][3])
        dealt.append(i)
    for x in splits:
        cuts.append((index[(x[0], x[1])], int(x[2]), int(x[3]), int(x[4]), int(x[5])))
    host.check_plan([t[3] for t in tiles], Hkv, grid, (shares, dealt, cuts, first))
    # the small tiles from the largest down, to a 256th of the largest that is not cut
    sizes = [tiles[i][3] for i in dealt]
    step = max(sizes, default=0) / 255 + 1
    assert all(b <= a + step for a, b in zip(sizes, sizes[1:]))
