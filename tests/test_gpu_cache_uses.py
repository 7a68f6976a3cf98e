"""The cache operators as programs use them beside each other: two calls at once, tables that share pages, graphs whose
inputs change between replays, batches that a plan cuts into shares.  Results are held against the oracle, with the
bounds that the parity tests derive, or bit for bit against the same call made alone."""

import numpy as np
import pytest

from oracle import cache as oc

from .helpers import torch_mod
from .test_gpu_cache import i32, np64, rotary_bound, turns_to_frequencies
from .test_gpu_cache_attn import SENTINEL, Attn
from .test_gpu_pages import bytes_of, make_caches, pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


@pytest.mark.parametrize("first,second", [
    (dict(q_len=[5, 2], kv_len=[3000, 700], D=128), dict(q_len=[60, 7], kv_len=[900, 2000], D=128)),
    (dict(q_len=[300], kv_len=[2500], D=64), dict(q_len=[1] * 9, kv_len=[400] * 9, D=64))])
def test_two_calls_at_once(sv, first, second):
    """Two streams, a workspace each, several rounds in flight: the bits of the calls made alone."""
    torch = torch_mod()
    problems = [Attn(append=True, seed=i, **kw) for i, kw in enumerate((first, second))]
    want = [c.run(sv)[0] for c in problems]
    after = [c.state() for c in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    outs, spaces = [], []
    for c in problems:
        c.to_device()
        outs.append([torch.full(c.q.shape, SENTINEL, device="cuda") for _ in range(6)])
        need = sv.spec_paged_attn8_workspace(c.d_q, c.d_codes[0], c.d_table, outs[-1][0], max_q=c.max_q)
        spaces.append(torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for i in range(6):  # the appends of all rounds write the same values
        for c, s, o, ws in zip(problems, streams, outs, spaces):
            sv.spec_paged_attn8(c.d_q, *c.d_codes, *c.d_exps, c.d_table, c.d_start, c.d_len, o[i], max_q=c.max_q,
                                k_new=c.d_new[0], v_new=c.d_new[1], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, w, o, ws, state in zip(problems, want, outs, spaces, after):
        assert sv.read_status(ws) == 0
        assert all(np.array_equal(np64(x), w) for x in o)
        assert all(np.array_equal(x, y) for x, y in zip(c.state(), state))


@pytest.mark.parametrize("q_len", [[2, 3, 1], [40, 12, 33]])
def test_rows_that_share_pages(sv, q_len):
    """A prefix that all rows have in common, and a page that one row holds three times."""
    c = Attn(q_len, [600, 512, 333], D=64, page=16, block=8, seed=3)
    c.table[1, :20] = c.table[0, :20]
    c.table[2, :12] = c.table[0, :12]
    c.table[1, 22] = c.table[1, 25] = c.table[1, 21]
    c.verify(sv)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 2)])
def test_many_sequences_cut_into_shares(sv, D, G):
    """Chunks, rounds, single tokens and resting sequences in one batch, whose long tiles several CTAs share."""
    rng = np.random.default_rng(D)
    q_len = [int(x) for x in rng.choice([0, 1, 1, 5, 26, 90, 160, 300], 24)]
    kv_len = [int(n + rng.integers(0 if n else 1, 3000)) for n in q_len]
    c = Attn(q_len, kv_len, D=D, G=G, page=32, append=True, seed=D)
    c.verify(sv, "bf16")


def test_rotary_captured(sv):
    """A graph of the call in place, replayed with other lengths, follows the rows that its call left."""
    torch = torch_mod()
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((20, 3, 64))).float().cuda()
    start, lens = i32([0, 7, 7, 19]), i32([900, 3, 12])
    steps, _ = sv.spec_rotary_steps(64)
    ws = torch.full((sv.spec_rotary_workspace(x, None, steps),), 255, dtype=torch.uint8, device="cuda")
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        sv.spec_rotary(x, None, steps, q_start=start, kv_len=lens, workspace=ws)
    f = turns_to_frequencies(steps)
    for new in ([900, 3, 12], [70000, 0, 40], [7, 1, 123456]):
        before = np64(x)
        lens.copy_(i32(new))
        g.replay()
        torch.cuda.synchronize()
        pos = np.concatenate([new[0] - 7 + np.arange(7), new[2] - 12 + np.arange(12), [0]])
        ref = oc.rotary(before, pos, f, False)
        ref[19] = before[19]
        assert np.all(np.abs(np64(x) - ref) <= rotary_bound(before, ref, 32, False, 1.0, "f32"))
        assert np.array_equal(np64(x)[19], before[19]) and sv.read_status(ws) == 0


def test_broadcast_rows_are_not_turned_in_place(sv):
    torch = torch_mod()
    x = torch.randn(1, 2, 64, device="cuda")
    steps, _ = sv.spec_rotary_steps(64)
    rows = x.expand(5, 2, 64)
    with pytest.raises(sv.SpecError):
        sv.spec_rotary(rows, None, steps, positions=i32(range(5)))
    out, _ = sv.spec_rotary(rows, None, steps, positions=i32(range(5)), q_out=torch.empty(5, 2, 64, device="cuda"))
    before = np64(rows)
    ref = oc.rotary(before, np.arange(5), turns_to_frequencies(steps), False)
    assert np.all(np.abs(np64(out) - ref) <= rotary_bound(before, ref, 32, False, 1.0, "f32"))


def test_compact_captured(sv):
    """Each replay compacts what the state holds by then; compacting twice moves nothing the second time."""
    torch = torch_mod()
    table, held, refs, rng = pool(700, 300, 12, 6)
    d_table, d_held, d_refs = i32(table), i32(held), i32(refs)
    caches = make_caches(700, rng)
    moved, live = i32(np.zeros(700)), i32([0])
    ws = torch.full((sv.spec_page_compact_workspace(d_table, d_refs),), 255, dtype=torch.uint8, device="cuda")
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        sv.spec_page_compact(d_table, d_held, d_refs, caches=caches, moved=moved, num_live=live, workspace=ws)
    for step in range(3):
        before = [bytes_of(c) for c in caches]
        table, refs = d_table.cpu().numpy(), d_refs.cpu().numpy()
        want = oc.page_compact(table, held, refs)
        assert step != 1 or not want[4]
        g.replay()
        torch.cuda.synchronize()
        assert sv.read_status(ws) == 0 and int(live) == want[3]
        assert np.array_equal(d_table.cpu().numpy(), want[0]) and np.array_equal(d_refs.cpu().numpy(), want[1])
        assert np.array_equal(moved.cpu().numpy(), want[2])
        for x, c in zip(before, caches):
            for src, dst in want[4]:
                x[dst] = x[src]
            assert np.array_equal(x, bytes_of(c))
        if step == 1:  # some pages are given back before the last replay
            gone = rng.choice(want[3], 40, replace=False)
            keep = ~np.isin(want[0], gone) & (np.arange(table.shape[1]) < held[:, None])
            t = np.zeros_like(table)
            for b in range(len(held)):
                r = want[0][b][keep[b]]
                held[b] = len(r)
                t[b, :len(r)] = r
            refs = want[1].copy()
            refs[gone] = 0
            d_table.copy_(i32(t))
            d_held.copy_(i32(held))
            d_refs.copy_(i32(refs))
