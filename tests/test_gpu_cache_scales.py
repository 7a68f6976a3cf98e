"""spec_paged_attn8 over block scales far apart: among 32 neighbouring keys, where the large one may be hidden from a row,
and from one end of the range to the other, where the normaliser has to count keys whose values hardly matter; and over
query rows that are not finite beside others.  Bounds are those of test_gpu_cache_attn.py: no scale of a neighbour enters them
but through W."""

import os

import numpy as np
import pytest

from oracle import cache as oc

from .helpers import torch_mod
from .test_gpu_cache import i32, np64
from .test_gpu_cache_attn import SENTINEL, Attn, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def blocks_of(c, tokens):
    """Indices (page, block) of these tokens of sequence 0."""
    tokens = np.asarray(tokens)
    return c.table[0, tokens // c.page], tokens % c.page // c.block


def in_few_rows(sv, c, ref, A, W, S):
    """The rows of a chunk again, in calls of up to 32 query rows per KV head."""
    torch = torch_mod()
    n, length, r0, most = int(c.start[1] - c.start[0]), int(c.kv_len[0]), int(c.start[0]), 32 // c.G
    for j in range(0, n, most):
        m = min(most, n - j)
        o = torch.full(c.q.shape, SENTINEL, device="cuda")
        sv.spec_paged_attn8(c.d_q, *c.d_codes, *c.d_exps, c.d_table, i32([r0 + j, r0 + j + m]), i32([length - n + j + m]), o,
                            max_q=m, window=c.window)
        rows = slice(r0 + j, r0 + j + m)
        check(np64(o)[rows], ref[rows], A[rows], W[rows], S, c.D, length, "f32", f"few rows from {j}")


@pytest.mark.parametrize("where", ["in view", "later", "before the window"])
@pytest.mark.parametrize("page,block", [(32, 1), (7, 7), (24, 24), (48, 24)])
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("gap", [15, 16, 24, 25, 26, 40, 120])
def test_a_large_neighbour(sv, gap, which, page, block, where):
    """Blocks 2^gap above their neighbours: once seen by all rows, once the chunk's last token, once the first that its
    first row sees.  What the other rows get does not depend on it.  Keys differ in a value that queries do not look at,
    so that the scores stay what they were."""
    D = 64 if gap % 2 else 128
    c = Attn([70], [300], G=4, Hkv=1, D=D, page=page, block=block, window=100 if where == "before the window" else 0,
             seed=gap + page)
    seen = range(300) if c.window == 0 else range(131, 300)
    tokens = {"in view": list(seen)[3::37], "later": [299], "before the window": [131]}[where]
    low = 120 if gap < 60 else 66
    r0, r1 = c.start[0], c.start[1]
    for i, e in enumerate(c.exps):
        far = which in ("kv"[i], "both")
        e[:] = c.rng.integers(low - 3, low + 1, e.shape) if far else c.rng.integers(117, 121, e.shape)
        if far:
            at = blocks_of(c, tokens)
            e[at[0], :, at[1]] = low + gap
            if i == 0:
                c.q[r0:r1] *= 2.0 ** (120 - low)
                c.q[r0:r1, :, 0] = 0.0
                big = np.zeros(c.codes[0].shape[2], bool)
                for page_id, blk in set(zip(*at)):
                    big[:] = False
                    big[blk * block:(blk + 1) * block] = True
                    k = c.codes[0][page_id][:, big]
                    k[..., 1:] = np.where(k[..., 1:] == 0x7F, 0x7F, 0)
                    c.codes[0][page_id][:, big] = k
    ref = c.reference()[0]
    c.verify(sv)
    in_few_rows(sv, c, *ref)


@pytest.mark.parametrize("q_len", [[5], [64]])
@pytest.mark.parametrize("seed", range(6))
def test_random_scales(sv, seed, q_len):
    """Scales of both kinds drawn per block from 2^-20 to 2^20, some of the blocks empty."""
    rng = np.random.default_rng(seed)
    page = int(rng.choice([8, 24, 32, 64]))
    block = int(rng.choice([b for b in (1, 2, 3, 4, 8, 12, 24, 32) if page % b == 0]))
    c = Attn(q_len, [int(rng.integers(70, 900))], G=4, Hkv=2, D=int(rng.choice([64, 128])), page=page, block=block,
             window=int(rng.choice([0, 40])), seed=seed)
    c.exps[1][:] = c.rng.integers(107, 148, c.exps[1].shape)
    empty = c.rng.random(c.exps[1].shape) < 0.2
    for x, e in zip(c.codes, c.exps):
        e[empty] = 63
        x[np.repeat(empty, block, axis=-1) & (x[..., 0] != 0x7F)] = 0
    c.exps[0][~empty] = c.rng.integers(90, 121, c.exps[0].shape)[~empty]
    c.verify(sv)


CALLS = int(os.environ.get("SPEC_RANDOM_CALLS", "30"))
SEED = int(os.environ.get("SPEC_RANDOM_SEED", "0"))


@pytest.mark.parametrize("seed", range(SEED, SEED + CALLS))
def test_random_calls_over_the_whole_range(sv, seed):
    """V's scales from 2^-64 to 2^64: any, a few of them, one far from the rest; K's large blocks differ in a value that
    queries do not look at."""
    rng = np.random.default_rng(12000 + seed)
    page = int(rng.choice([1, 7, 16, 24, 32, 64]))
    block = int(rng.choice([b for b in range(1, page + 1) if page % b == 0]))
    most = int(rng.choice([8, 60, 200]))
    q = [int(rng.integers(1, most + 1)) for _ in range(int(rng.choice([1, 2, 5])))]
    c = Attn(q, [n + int(2 ** rng.uniform(0, 11)) for n in q], G=int(rng.choice([1, 4])), Hkv=int(rng.choice([1, 2])),
             D=int(rng.choice([64, 128])), page=page, block=block, window=int(rng.choice([0, 0, 30])),
             append=bool(rng.random() < 0.3), seed=seed)
    lo, hi = sorted(int(x) for x in rng.integers(63, 192, 2))
    e = c.exps[1]
    e[:] = (c.rng.integers(lo, hi + 1, e.shape) if seed % 4 < 2 else c.rng.choice([63, 127, 191], e.shape) if seed % 4 == 2 else
            np.where(c.rng.random(e.shape) < 0.05, hi, lo))
    if seed % 4 != 1 and not c.do_append:
        r0, r1 = c.start[0], c.start[-1]
        low = int(rng.integers(66, 130))
        far = c.rng.random(c.exps[0].shape) < 0.1
        c.exps[0][:] = np.where(far, min(low + int(rng.integers(0, 120)), 191), low - c.rng.integers(0, 3, far.shape))
        c.q[r0:r1] *= 2.0 ** (120 - low)
        c.q[r0:r1, :, 0] = 0.0
        codes = c.codes[0]
        hidden = np.repeat(far, block, axis=-1)[..., None] & (codes != 0x7F)
        hidden[..., 0] = False
        codes[hidden] = 0
    c.verify(sv, what=f"seed {seed}", max_q=int(rng.choice([c.max_q, c.max_q + 40])))


def rising(c, codes, byte):
    """Keys of sequence 0 whose score with a row (1, 0, 0, ...) is what `codes` says, times 2^(byte - 127)."""
    c.q[:] = 0.0
    c.q[:, :, 0] = 1.0
    for t, code in enumerate(codes):
        page, slot = c.table[0, t // c.page], t % c.page
        c.codes[0][page, :, slot] = 0
        c.codes[0][page, :, slot, 0] = code
    c.exps[0][:] = byte


@pytest.mark.parametrize("order", ["falling", "rising", "mixed"])
@pytest.mark.parametrize("q,length", [(2, 300), (3, 9000), (60, 300), (60, 5000)])
def test_normaliser_over_the_whole_range(sv, q, length, order):
    """Equal scores, and V's scales from 2^-64 to 2^64: values of the smallest do not show beside the largest, but their
    keys count as much.  In one tile, in several, in the shares of several CTAs."""
    c = Attn([q], [length], G=4, Hkv=2, D=64 if q % 2 else 128, page=32, block=32, seed=q)
    rising(c, [0] * length, 127)
    t = np.arange(length) // 32
    last = t[-1]
    byte = {"falling": np.where(t == 0, 191, 63), "rising": np.where(t == last, 191, 63),
            "mixed": np.where(t == last // 2, 191, np.where(t % 3 == 1, 66, 63))}[order]
    c.exps[1][c.table[0, t], :, 0] = byte[:, None]
    c.verify(sv)


@pytest.mark.parametrize("block", [1, 8, 32])
@pytest.mark.parametrize("q,length", [(2, 700), (60, 700), (64, 4000)])
@pytest.mark.parametrize("steps", [4, 10, 16])
def test_normaliser_of_unequal_scores(sv, q, length, block, steps):
    """The keys of large scale have scores above the others', by up to 2^steps in the weight: what is counted of the small
    ones lies far below the range of the products."""
    c = Attn([q], [length], G=2, Hkv=1, D=64, page=32, block=block, seed=q + steps)
    at, blk = blocks_of(c, np.arange(length))
    large = c.rng.random(c.exps[1].shape) < 0.03
    large[c.table[0, 0]] = True
    big = large[at, 0, blk]
    rising(c, np.where(big, 0x38, 0), 127)         # scores 1 and 0, times scale
    c.exps[1][:] = np.where(large, 191, 66)
    ln2 = float(np.log(2.0))
    ref, A, W, S = oc.paged_attn8(
        np64(c.q), c.codes, c.exps, c.table, c.start, c.kv_len, 0, steps * ln2)
    o, st = c.run(sv, scale=steps * ln2)
    r0, r1 = c.start[0], c.start[1]
    assert st == 0
    check(o[r0:r1], ref[r0:r1], A[r0:r1], W[r0:r1], S, 64, length, "f32")


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), 2.0 ** 126])
@pytest.mark.parametrize("q,length", [(1, 200), (5, 200), (5, 9000), (60, 200)])
def test_a_row_that_is_not_finite_is_alone(sv, q, length, value):
    """A query row that is not finite, or too large, leaves the other rows as they are, those of its token and KV head too."""
    c = Attn([q], [length], G=4, Hkv=2, D=64, seed=9)
    ref, A, W, S = c.reference()[0]
    r0, r1 = int(c.start[0]), int(c.start[1])
    c.q[r0 + q // 2, 5, 7] = value
    o, st = c.run(sv)
    keep = np.ones((q, 8), bool)
    keep[q // 2, 5] = False
    assert st == 0
    check(o[r0:r1][keep], ref[r0:r1][keep], A[r0:r1][keep], W[r0:r1][keep], S, 64, length, "f32")
