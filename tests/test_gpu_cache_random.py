"""Random calls of the cache operators against their oracles, with seeds.  SPEC_RANDOM_CALLS and SPEC_RANDOM_SEED make
more of them."""

import os

import numpy as np
import pytest

from oracle import cache as oc

from .helpers import torch_mod
from .test_gpu_cache import Cache8, i32, np64, rotary_bound, turns_to_frequencies
from .test_gpu_cache_attn import Attn
from .test_gpu_pages import Beams, bytes_of, pool

pytestmark = pytest.mark.gpu

CALLS = int(os.environ.get("SPEC_RANDOM_CALLS", "30"))
SEED = int(os.environ.get("SPEC_RANDOM_SEED", "0"))


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def batch(rng, most_rows, most_tokens):
    """Lengths of a ragged batch: resting sequences, first tokens, chunks of prompts."""
    B = int(rng.choice([1, 2, 3, 7, 40]))
    top = int(2 ** rng.uniform(0, np.log2(most_rows)))
    q = [0 if rng.random() < 0.1 else int(rng.integers(1, top + 1)) for _ in range(B)]
    q[0] = max(q[0], 1)
    old = [0 if rng.random() < 0.2 else int(2 ** rng.uniform(0, np.log2(most_tokens / (1 + B // 8)))) for _ in range(B)]
    return q, [max(a + b, 1) for a, b in zip(q, old)]


def cache_of(rng):
    page = int(rng.choice([1, 7, 16, 24, 32, 64, 128]))
    blocks = [b for b in range(1, page + 1) if page % b == 0]
    return dict(page=page, block=int(rng.choice(blocks)), D=int(rng.choice([64, 128])), Hkv=int(rng.integers(1, 4)),
                layout=str(rng.choice(["hnd", "nhd"])), lead=int(rng.integers(0, 3)), trail=int(rng.integers(0, 3)))


@pytest.mark.parametrize("seed", range(SEED, SEED + CALLS))
def test_random_attention(sv, seed):
    rng = np.random.default_rng(7000 + seed)
    kw = cache_of(rng)
    G = int(rng.choice([1, 2, 4, 8, 32]))
    q, kv = batch(rng, max(1, int(rng.choice([32, 300])) // G), 2500)
    window = int(rng.choice([0, 0, 1, 20, 300]))
    exps = dict(exp_lo=int(rng.integers(100, 118)), exp_hi=120)
    exps["exp_lo"] = max(exps["exp_lo"], 116) if rng.random() < 0.7 else exps["exp_lo"]
    # scales more than 2^14 apart among 32 keys would lose bits of small values in large chunks
    exps["exp_lo"] = max(exps["exp_lo"], 110)
    c = Attn(q, kv, G=G, window=window, append=bool(rng.random() < 0.5), seed=seed, **kw, **exps)
    o = c.verify(sv, "bf16" if rng.random() < 0.3 else "f32", what=f"seed {seed}", max_q=int(rng.choice([c.max_q, c.max_q + 50])))
    assert np.all(np.isfinite(o[c.start[0]:c.start[-1]]))


@pytest.mark.parametrize("seed", range(SEED, SEED + CALLS))
def test_random_append(sv, seed):
    rng = np.random.default_rng(8000 + seed)
    q, kv = batch(rng, 700, 1500)
    c = Cache8(q, kv, dtype=str(rng.choice(["bf16", "f32"])), seed=seed, scale=2.0 ** int(rng.integers(-70, 70)), **cache_of(rng))
    for x in c.new:  # a few values that are not finite
        flat = x.view(-1)
        at = rng.integers(0, flat.numel(), 5)
        flat[at] = flat.new_tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0])
    c.verify(sv)


@pytest.mark.parametrize("seed", range(SEED, SEED + CALLS))
def test_random_rotary(sv, seed):
    torch = torch_mod()
    rng = np.random.default_rng(9000 + seed)
    dtype = str(rng.choice(["bf16", "f32"]))
    T, H, D = int(2 ** rng.uniform(0, 10)), int(rng.integers(1, 9)), int(rng.choice([8, 64, 80, 128, 256]))
    rot = 2 * int(rng.integers(1, D // 2 + 1)) if rng.random() < 0.6 else D
    pairs, inverse = bool(rng.random() < 0.5), bool(rng.random() < 0.3)
    x = torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    pos = rng.integers(-1000, int(2 ** rng.uniform(4, 31)), T)
    steps, _ = sv.spec_rotary_steps(rot, float(rng.choice([10000.0, 500000.0])), kind=sv.SPEC_ROTARY_LINEAR, factor=float(rng.choice([1, 3.7])))
    amp = float(np.float32(rng.choice([1.0, 1.13])))
    x0 = np64(x)
    out = None if rng.random() < 0.5 else torch.zeros_like(x)
    y, _ = sv.spec_rotary(x, None, steps, positions=i32(pos), q_out=out, amplitude=amp, inverse=inverse,
                          layout=sv.SPEC_ROTARY_PAIRS if pairs else sv.SPEC_ROTARY_HALF)
    ref = oc.rotary(x0, pos, turns_to_frequencies(steps), pairs, amp, inverse)
    assert np.all(np.abs(np64(y) - ref) <= rotary_bound(x0, ref, rot // 2, pairs, amp, dtype))


@pytest.mark.parametrize("seed", range(SEED, SEED + CALLS))
def test_random_fork(sv, seed):
    rng = np.random.default_rng(10000 + seed)
    B = int(2 ** rng.uniform(0, 9))
    b = Beams(B, int(rng.choice([1, 3, 16, 64])), int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 11)), seed,
              int(rng.integers(0, 40)), drop=float(rng.choice([0, 0.2, 0.9])), spread=bool(rng.random() < 0.8))
    b.verify(sv, bool(rng.random() < 0.5), grow=bool(rng.random() < 0.9))


@pytest.mark.parametrize("seed", range(SEED, SEED + CALLS))
def test_random_compact(sv, seed):
    torch = torch_mod()
    rng = np.random.default_rng(11000 + seed)
    pages = int(2 ** rng.uniform(0, 14))
    table, held, refs, rng = pool(pages, int(rng.integers(0, pages + 1)), int(2 ** rng.uniform(0, 7)), seed)
    want = oc.page_compact(table, held, refs)
    caches = [torch.from_numpy(rng.integers(0, 256, (pages, n)).astype(np.uint8)).cuda() for n in (48, int(rng.integers(1, 40)))]
    before = [bytes_of(c) for c in caches]
    moved = i32(np.zeros(pages))
    t, r = sv.spec_page_compact(i32(table), i32(held), i32(refs), caches=caches, moved=moved)
    for got, ref in zip((t, r, moved), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    for x, c in zip(before, caches):
        for src, dst in want[4]:
            x[dst] = x[src]
        assert np.array_equal(x, bytes_of(c))
