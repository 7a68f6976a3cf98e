"""GPU parity of spec_page_fork and spec_page_compact against the step-by-step oracle, bit for bit, pages' contents
included."""

import numpy as np
import pytest

from oracle import cache as oc

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def i32(x):
    torch = torch_mod()
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def make_caches(pages, rng):
    """Arrays of all kinds: whole 16s, odd sizes, a page of several pieces, one inside a wider buffer."""
    torch = torch_mod()
    raw = lambda *s: torch.from_numpy(rng.integers(0, 256, (pages, *s)).astype(np.uint8)).cuda()  # noqa: E731
    return [raw(2, 16, 64).view(torch.bfloat16), raw(3), raw(1, 7, 5), raw(40, 1024), raw(2, 48)[:, 1],
            raw(2, 16, 8, 16).permute(0, 2, 1, 3, 4)]


def bytes_of(c):
    torch = torch_mod()
    return c.contiguous().view(torch.uint8).cpu().numpy().reshape(c.shape[0], -1)


class Beams:
    """Rows that share pages at random, with external holders."""

    def __init__(self, B, page, top, spare, seed, grow_to=6, drop=0.2, spread=True):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.page = B, page
        rows, self.kv_len, nxt = [], [], 0
        for b in range(B):
            if b and rng.random() < 0.5:  # a fork of an earlier row: all, or all but the last page
                src = int(rng.integers(0, b))
                r, n = list(rows[src]), self.kv_len[src]
                if r and rng.random() < 0.5:
                    r[-1] = nxt
                    nxt += 1
            else:
                n = int(rng.integers(0, top + 1))
                r = list(range(nxt, nxt + -(-n // page)))
                nxt += len(r)
            rows.append(r)
            self.kv_len.append(n)
        for b in range(B):  # pages past the tokens, from a rollback
            if rng.random() < 0.3:
                rows[b] = rows[b] + [nxt]
                nxt += 1
        self.pages = max(nxt + spare, 1)
        order = rng.permutation(self.pages)
        cols = max(max(len(r) for r in rows), 1) + grow_to // page + 2
        self.table = rng.integers(-5, 5, (B, cols)).astype(np.int32)
        refs = np.zeros(self.pages, np.int32)
        for b, r in enumerate(rows):
            self.table[b, :len(r)] = order[r]
            for e in order[r]:
                refs[e] += 1
        refs[rng.random(self.pages) < 0.05] += 1
        self.refs = refs
        self.held = np.array([len(r) for r in rows], np.int32)
        self.kv_len = np.array(self.kv_len, np.int32)
        self.parent = np.where(rng.random(B) < drop, -1, rng.integers(0, B, B) if spread else np.arange(B)).astype(np.int32)
        self.grow = rng.integers(0, grow_to + 1, B).astype(np.int32)

    def run(self, sv, in_place, grow=True, caches=None, stream=None):
        torch = torch_mod()
        state = [i32(x) for x in (self.table, self.held, self.kv_len, self.refs)]
        outs = {} if in_place else dict(zip(("table_out", "held_out", "len_out", "refs_out"), [x.clone() for x in state]))
        caches = make_caches(self.pages, self.rng) if caches is None else caches
        before = [bytes_of(c) for c in caches]
        ws = torch.full((sv.spec_page_fork_workspace(state[0], state[3]),), 255, dtype=torch.uint8, device="cuda")
        got = sv.spec_page_fork(*state, i32(self.parent), page_size=self.page, grow=i32(self.grow) if grow else None,
                                caches=caches, workspace=ws, **outs)
        torch.cuda.synchronize()
        if not in_place:
            for x, y in zip(state, (self.table, self.held, self.kv_len, self.refs)):
                assert np.array_equal(x.cpu().numpy(), y)
        return [x.cpu().numpy() for x in got], before, [bytes_of(c) for c in caches], sv.read_status(ws)

    def verify(self, sv, in_place, grow=True):
        want = oc.page_fork(self.table, self.held, self.kv_len, self.refs, self.parent, self.grow if grow else [0] * self.B, self.page)
        got, before, after, status = self.run(sv, in_place, grow)
        if want is None:
            assert status == sv.SPEC_STATUS_NO_PAGE
            want = (self.table, self.held, self.kv_len, self.refs, [])
        else:
            assert status == 0
        for name, a, b in zip(("table", "held", "kv_len", "refs"), got, want):
            assert np.array_equal(a, b), name
        for x in before:
            for src, dst in want[4]:
                x[dst] = x[src]
        assert all(np.array_equal(a, b) for a, b in zip(before, after))
        return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,top,spare,grow_to", [
    (1, 16, 0, 0, 0), (1, 16, 5, 3, 20), (2, 1, 9, 40, 3), (8, 16, 100, 60, 6), (37, 4, 300, 600, 9), (64, 64, 900, 300, 1),
    (200, 16, 700, 900, 40), (1100, 16, 90, 5000, 17), (4096, 2, 5, 40000, 5), (5, 1, 700, 100, 2), (30, 16, 200, 10, 40)])
def test_fork_parity(sv, B, page, top, spare, grow_to, in_place):
    for seed in range(3):
        Beams(B, page, top, spare, 100 * seed + B, grow_to).verify(sv, in_place)


def test_fork_reports_too_few_pages(sv):
    """The last of these batches' free pages decides."""
    b = Beams(20, 16, 200, 200, 5, 40)
    want = b.verify(sv, True)
    used = int((want[3] > 0).sum())
    assert used < b.pages
    # free pages that others hold now: exactly enough, then one too few
    freed = [i for i in range(b.pages) if want[3][i] <= 0]
    b.refs[freed] += 1
    assert b.verify(sv, False)[4] == want[4]
    first_new = int(next(i for i in range(b.pages) if want[3][i] > 0 and b.refs[i] <= 0))
    b.refs[first_new] = 1
    assert b.verify(sv, True)[4] == []


def test_fork_rows_that_stay_and_rows_without_growth(sv):
    for kw in (dict(drop=0.0, spread=False), dict(drop=1.0), dict(drop=0.3)):
        Beams(50, 16, 300, 300, 7, 5, **kw).verify(sv, True)
        Beams(50, 16, 300, 0, 8, 5, **kw).verify(sv, True, grow=False)


def test_fork_last_holder_keeps_its_page(sv):
    """Four rows from one parent whose last page nobody else keeps: the lowest row keeps it, three copies are made."""
    b = Beams(4, 16, 40, 20, 11, 5)
    b.table[:, :3] = np.array([[0, 1, 2], [3, 4, 5], [6, 7, 8], [9, 10, 11]])
    b.held[:], b.kv_len[:], b.grow[:], b.parent[:] = 3, 40, 1, 2
    b.refs[:] = 0
    b.refs[:12] = 1
    want = b.verify(sv, True)
    assert want[4] == [(8, 0), (8, 1), (8, 2)] and want[0][0, 2] == 8
    b.refs[8] = 2  # and somebody else: all copy
    assert len(b.verify(sv, False)[4]) == 4


@pytest.mark.parametrize("what,flag", [
    (dict(parent=-2), 16), (dict(parent=6), 16), (dict(kv_len=-1), 1), (dict(kv_len=1000), 1), (dict(held=-1), 1),
    (dict(held=99), 1), (dict(grow=-1), 1), (dict(grow=2 ** 31 - 1), 1), (dict(table=-1), 32), (dict(table=10 ** 6), 32)])
def test_fork_bad_data_changes_nothing(sv, what, flag):
    b = Beams(6, 16, 100, 50, 3, 5, drop=0.0)
    b.parent = np.array([1, 0, 2, 3, 3, 5], np.int32)
    b.kv_len[:], b.held[:] = 20, 2
    b.table[:, :2] = np.arange(12).reshape(6, 2)
    b.refs[:] = (np.arange(b.pages) < 12)
    (name, value), = what.items()
    if name == "table":
        b.table[3, 1] = value
    else:
        getattr(b, name)[3] = value
    for in_place in (True, False):
        got, before, after, status = b.run(sv, in_place)
        assert status == flag
        for a, ref in zip(got, (b.table, b.held, b.kv_len, b.refs)):
            assert np.array_equal(a, ref)
        assert all(np.array_equal(x, y) for x, y in zip(before, after))


def test_fork_many_arrays(sv):
    """More arrays than one launch of the copies takes."""
    torch = torch_mod()
    b = Beams(12, 16, 100, 60, 21, 5, drop=0.0)
    caches = [torch.from_numpy(b.rng.integers(0, 256, (b.pages, 16 + i)).astype(np.uint8)).cuda() for i in range(101)]
    want = oc.page_fork(b.table, b.held, b.kv_len, b.refs, b.parent, b.grow, b.page)
    assert want[4]
    got, before, after, status = b.run(sv, True, caches=caches)
    assert status == 0 and np.array_equal(got[0], want[0])
    for x, y in zip(before, after):
        for src, dst in want[4]:
            x[dst] = x[src]
        assert np.array_equal(x, y)


def test_fork_captured_in_place(sv):
    """A decoding loop's step as a graph: every replay goes on from the state that the one before left."""
    torch = torch_mod()
    b = Beams(9, 4, 30, 200, 33, 3, drop=0.0)
    state = [i32(x) for x in (b.table, b.held, b.kv_len, b.refs)]
    wide = i32(np.pad(b.table, ((0, 0), (0, 20))))
    state[0] = wide
    parent, grow = i32(b.parent), i32(b.grow)
    caches = make_caches(b.pages, b.rng)
    ws = torch.zeros(sv.spec_page_fork_workspace(wide, state[3]), dtype=torch.uint8, device="cuda")
    host = [x.cpu().numpy() for x in state]
    held_bytes = [bytes_of(c) for c in caches]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        sv.spec_page_fork(*state, parent, page_size=4, grow=grow, caches=caches, workspace=ws)
    for step in range(6):
        p, n = b.rng.integers(-1, 9, 9).astype(np.int32), b.rng.integers(0, 4, 9).astype(np.int32)
        p[0], p[1] = step % 9, -1
        parent.copy_(i32(p))
        grow.copy_(i32(n))
        g.replay()
        torch.cuda.synchronize()
        want = oc.page_fork(*host, p, n, 4)
        assert want is not None and sv.read_status(ws) == 0
        host = list(want[:4])
        for x, y in zip(state, host):
            assert np.array_equal(x.cpu().numpy(), y), step
        for x, c in zip(held_bytes, caches):
            for src, dst in want[4]:
                x[dst] = x[src]
            assert np.array_equal(x, bytes_of(c))


# ------------------------------------------------------------------------------ compact
def pool(pages, live, rows, seed, cols_extra=2):
    rng = np.random.default_rng(seed)
    used = rng.permutation(pages)[:live]
    refs = np.zeros(pages, np.int32)
    refs[used] = rng.integers(1, 4, live)
    refs[rng.random(pages) < 0.02 * (refs == 0)] = -1
    held = rng.integers(0, max(1, min(live, 40)) + 1, rows).astype(np.int32) if live else np.zeros(rows, np.int32)
    table = rng.integers(-9, 10 ** 6, (rows, int(held.max(initial=0)) + cols_extra)).astype(np.int32)
    for b in range(rows):
        table[b, :held[b]] = rng.choice(used, held[b]) if held[b] else table[b, :0]
    return table, held, refs, rng


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pages,live,rows", [(1, 0, 1), (1, 1, 1), (7, 3, 2), (31, 30, 4), (33, 1, 3), (1000, 500, 17), (1000, 0, 2),
                                             (1000, 1000, 5), (2500, 2400, 300), (40000, 30000, 64), (70000, 100, 9)])
def test_compact_parity(sv, pages, live, rows, in_place):
    torch = torch_mod()
    table, held, refs, rng = pool(pages, live, rows, pages + live)
    want = oc.page_compact(table, held, refs)
    d_table, d_held, d_refs = i32(table), i32(held), i32(refs)
    outs = {} if in_place else dict(table_out=d_table.clone(), refs_out=torch.full_like(d_refs, 77))
    caches = make_caches(pages, rng) if pages <= 2500 else [torch.from_numpy(rng.integers(0, 256, (pages, n)).astype(np.uint8)).cuda() for n in (64, 5)]
    before = [bytes_of(c) for c in caches]
    moved, live_out = i32(np.full(pages, 5)), i32([-1])
    ws = torch.full((sv.spec_page_compact_workspace(d_table, d_refs),), 255, dtype=torch.uint8, device="cuda")
    t, r = sv.spec_page_compact(d_table, d_held, d_refs, caches=caches, moved=moved, num_live=live_out, workspace=ws, **outs)
    torch.cuda.synchronize()
    assert sv.read_status(ws) == 0
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(r.cpu().numpy(), want[1])
    assert np.array_equal(moved.cpu().numpy(), want[2]) and int(live_out) == want[3]
    for x, c in zip(before, caches):
        for src, dst in want[4]:
            x[dst] = x[src]
        assert np.array_equal(x, bytes_of(c))


@pytest.mark.parametrize("bad,flag", [("held", 1), ("low", 32), ("high", 32), ("free", 32)])
def test_compact_bad_data_changes_nothing(sv, bad, flag):
    torch = torch_mod()
    table, held, refs, rng = pool(500, 200, 8, 4)
    held[3] = 5
    table[3, :5] = np.flatnonzero(refs > 0)[:5]
    if bad == "held":
        held[3] = table.shape[1] + 1
    else:
        table[3, 2] = {"low": -1, "high": 500, "free": np.flatnonzero(refs <= 0)[0]}[bad]
    d = [i32(x) for x in (table, held, refs)]
    caches = make_caches(500, rng)
    before = [bytes_of(c) for c in caches]
    ws = torch.zeros(sv.spec_page_compact_workspace(d[0], d[2]), dtype=torch.uint8, device="cuda")
    moved = i32(np.full(500, 5))
    sv.spec_page_compact(*d, caches=caches, moved=moved, workspace=ws)
    torch.cuda.synchronize()
    assert sv.read_status(ws) == flag
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(d, (table, held, refs)))
    assert all(np.array_equal(x, bytes_of(c)) for x, c in zip(before, caches)) and bool((moved == 5).all())


def test_compact_without_caches_and_outputs(sv):
    table, held, refs, _ = pool(300, 100, 6, 1)
    want = oc.page_compact(table, held, refs)
    t, r = sv.spec_page_compact(i32(table), i32(held), i32(refs))
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(r.cpu().numpy(), want[1])


def test_page_calls_on_another_stream(sv):
    torch = torch_mod()
    side = torch.cuda.Stream()
    b = Beams(20, 16, 100, 100, 41, 5)
    want = oc.page_fork(b.table, b.held, b.kv_len, b.refs, b.parent, b.grow, 16)
    state = [i32(x) for x in (b.table, b.held, b.kv_len, b.refs)]
    parent, grow = i32(b.parent), i32(b.grow)
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_page_fork(*state, parent, page_size=16, grow=grow, stream=side)
    compacted = sv.spec_page_compact(got[0], got[1], got[3], stream=side)
    side.synchronize()
    t, r, *_ = oc.page_compact(want[0], want[1], want[3])
    assert np.array_equal(compacted[0].cpu().numpy(), t) and np.array_equal(compacted[1].cpu().numpy(), r)
