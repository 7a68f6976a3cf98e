"""The cache operators without a workspace, on the current stream and on another at once: neither takes memory that the
other still uses, and both give what they give alone, bit for bit."""

import pytest

from .helpers import torch_mod
from .test_gpu_cache import i32
from .test_gpu_cache_attn import Attn
from .test_gpu_pages import Beams, make_caches, pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def attention(sv, seed, q_len, kv_len, append):
    torch = torch_mod()
    c = Attn(q_len, kv_len, D=128, append=append, seed=seed).to_device()
    q = c.q.cuda()
    new = dict(k_new=c.d_new[0], v_new=c.d_new[1]) if append else {}
    out = torch.zeros(q.shape, device="cuda")
    need = sv.spec_paged_attn8_workspace(q, c.d_codes[0], c.d_table, out, max_q=c.max_q)

    def call(stream=None):
        sv.spec_paged_attn8(q, *c.d_codes, *c.d_exps, c.d_table, c.d_start, c.d_len, out, max_q=c.max_q, stream=stream, **new)
        return [out[c.start[0]:c.start[-1]], *(x.view(torch.uint8) for x in (*c.d_codes, *c.d_exps))]

    return call, need


def append(sv, seed):
    torch = torch_mod()
    c = Attn([40, 7, 0, 300], [60, 500, 9, 300], D=64, append=True, seed=seed).to_device()

    def call(stream=None):
        sv.spec_kv8_append(*c.d_new, *c.d_codes, *c.d_exps, c.d_table, c.d_start, c.d_len, stream=stream)
        return [x.view(torch.uint8) for x in (*c.d_codes, *c.d_exps)]

    return call, sv.spec_kv8_append_workspace(c.d_new[0], c.d_table)


def rotary(sv, seed):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = (torch.randn(500, h, 64, generator=g, device="cuda") for h in (4, 2))
    steps, _ = sv.spec_rotary_steps(64)
    pos = torch.randint(0, 10 ** 6, (500,), generator=g, device="cuda", dtype=torch.int32)
    outs = torch.zeros_like(q), torch.zeros_like(k)
    call = lambda stream=None: list(sv.spec_rotary(q, k, steps, positions=pos, q_out=outs[0], k_out=outs[1], stream=stream))  # noqa: E731
    return call, sv.spec_rotary_workspace(q, k, steps)


def fork(sv, seed):
    b = Beams(60, 16, 300, 600, seed, 20)
    state = [i32(x) for x in (b.table, b.held, b.kv_len, b.refs)]
    outs = dict(zip(("table_out", "held_out", "len_out", "refs_out"), [x.clone() for x in state]))
    parent, grow, caches = i32(b.parent), i32(b.grow), make_caches(b.pages, b.rng)
    call = lambda stream=None: list(sv.spec_page_fork(*state, parent, page_size=16, grow=grow, caches=caches, stream=stream, **outs))  # noqa: E731
    return call, sv.spec_page_fork_workspace(state[0], state[3])


def compact(sv, seed):
    torch = torch_mod()
    table, held, refs, rng = pool(900, 400, 30, seed)
    d = [i32(x) for x in (table, held, refs)]
    outs = dict(table_out=d[0].clone(), refs_out=d[2].clone(), moved=torch.zeros_like(d[2]))
    call = lambda stream=None: [*sv.spec_page_compact(*d, caches=make, stream=stream, **outs), outs["moved"]]  # noqa: E731
    make = make_caches(900, rng)
    return call, sv.spec_page_compact_workspace(d[0], d[2])


CALLS = {
    "few rows": lambda sv, seed: attention(sv, seed, [4, 1], [9000, 5000], False),
    "few rows, append": lambda sv, seed: attention(sv, seed, [4, 1], [9000, 5000], True),
    "chunks": lambda sv, seed: attention(sv, seed, [300, 40], [4000, 2500], False),
    "chunks, append": lambda sv, seed: attention(sv, seed, [300, 40], [4000, 2500], True),
    "append": append, "rotary": rotary, "fork": fork, "compact": compact,
}


@pytest.mark.parametrize("name", CALLS)
def test_current_stream_and_given_stream_at_once(sv, name):
    torch = torch_mod()
    one, two = (CALLS[name](sv, seed)[0] for seed in (1, 2))
    want = [[x.clone() for x in call()] for call in (one, two)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        torch.cuda.synchronize()
        one()
        b = two(stream=side)
        a = one()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, want[0])) and all(torch.equal(x, y) for x, y in zip(b, want[1]))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_a_dropped_tensor_still_being_read(sv, name, raw):
    """A temporary of the current stream, dropped while a copy of it waits there: the call on the other stream (an object
    or its raw handle) does not write to it."""
    torch = torch_mod()
    call, need = CALLS[name](sv, 3)
    want = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temp = torch.full((need,), 3, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    seen = temp.clone()
    del temp
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert bool((seen == 3).all()) and all(torch.equal(x, y) for x, y in zip(got, want))
