"""Calls with stream= and no workspace beside work of the current stream: neither takes memory that the other
still uses, and both give what they give alone, bit for bit."""

import pytest

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def paged(sv, seed, q_len, kv_len, dtype):
    """spec_paged_attn on inputs of its own: call(out, **kw), bytes of workspace, a new output."""
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, Hq, Hkv, D, page = len(q_len), 8, 2, 128, 32
    norm = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cols = -(-max(kv_len) // page)
    q, k, v = norm(sum(q_len), Hq, D), norm(B * cols, Hkv, page, D), norm(B * cols, Hkv, page, D)
    table = torch.randperm(B * cols, generator=g, device="cuda").to(torch.int32).view(B, cols)
    start, lens = i32([sum(q_len[:b]) for b in range(B + 1)]), i32(kv_len)
    need = sv.spec_paged_attn_workspace(q, k, table, q, max_q=max(q_len))
    call = lambda out, **kw: sv.spec_paged_attn(q, k, v, table, start, lens, out, max_q=max(q_len), **kw)  # noqa: E731
    return call, need, lambda: torch.zeros(q.shape, device="cuda")


def prefill(sv, seed, lens):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    q, k, v = (torch.randn(T, h, 64, generator=g, device="cuda").to(torch.bfloat16) for h in (8, 2, 2))
    start = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    need = sv.spec_prefill_attn_workspace(q, k, start, q)
    return (lambda out, **kw: sv.spec_prefill_attn(q, k, v, start, out, **kw)), need, lambda: torch.zeros(
        q.shape, device="cuda")


def logprobs(sv, seed, N):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, 50257, generator=g, device="cuda")
    tok = torch.randint(0, 50257, (N,), generator=g, device="cuda", dtype=torch.int32)
    need = sv.spec_token_logprobs_workspace(x, 0)
    return (lambda out, **kw: sv.spec_token_logprobs(x, tok, out, **kw)), need, lambda: torch.zeros(N, device="cuda")


CALLS = {
    "paged-split": lambda sv, seed: paged(sv, seed, [4, 1], [30000, 20000], "bf16"),
    "paged-chunk": lambda sv, seed: paged(sv, seed, [300, 40], [9000, 5000], "bf16"),
    "paged-fp32": lambda sv, seed: paged(sv, seed, [30, 4], [2000, 500], "f32"),
    "prefill": lambda sv, seed: prefill(sv, seed, [900, 1500, 40]),
    "logprobs": lambda sv, seed: logprobs(sv, seed, 5),
}


@pytest.mark.parametrize("name", CALLS)
def test_current_stream_and_given_stream_at_once(sv, name):
    torch = torch_mod()
    (one, _, out1), (two, _, out2) = CALLS[name](sv, 1), CALLS[name](sv, 2)
    want = one(out=out1()).clone(), two(out=out2()).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        a, b = out1(), out2()
        torch.cuda.synchronize()
        one(out=a)
        two(out=b, stream=side)
        one(out=a)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_a_dropped_tensor_still_being_read(sv, name, raw):
    """A temporary of the current stream, dropped while a copy of it waits there: the call on the other
    stream (an object or its raw handle) does not write to it."""
    torch = torch_mod()
    call, need, out = CALLS[name](sv, 3)
    want = call(out=out()).clone()
    o, side = out(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temp = torch.full((need,), 3, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    seen = temp.clone()
    del temp
    call(out=o, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert bool((seen == 3).all()) and torch.equal(o, want)


def round_calls(sv):
    """The calls of the speculative round: name -> (call(stream) -> outputs, bytes of workspace)."""
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(9)
    norm = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    b16 = lambda *s: norm(*s).to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v, lens = b16(2, 5, 8, 128), b16(2, 2, 4096, 128), b16(2, 2, 4096, 128), i32([4000, 1500])
    wq, wk, wv, pos = b16(2, 8, 128), b16(2, 2, 512, 128), b16(2, 2, 512, 128), i32([700, 300])
    logits, hidden, weight = norm(2, 5, 32000), b16(2, 5, 256), b16(32000, 256)
    drafts = torch.randint(0, 32000, (2, 4), generator=g, device="cuda", dtype=torch.int32)
    o, wo = torch.empty((2, 5, 8, 128), device="cuda"), torch.empty((2, 8, 128), device="cuda")
    tok, acc = torch.empty((2, 5), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    none, mode = i32([0, 0]), sv.SPEC_SAMPLE_CHAIN_GREEDY
    return {
        "verify": (lambda s: [sv.spec_verify_attn(q, k, v, lens, o, stream=s)], sv.spec_verify_attn_workspace(q, k, o)),
        "window": (lambda s: [sv.spec_draft_window_attn(wq, wk, wv, pos, wo, stream=s)],
                   sv.spec_draft_window_attn_workspace(wq, wk, wo)),
        "sample": (lambda s: sv.spec_sample(mode, logits, tok, acc, draft_tokens=drafts, stream=s),
                   sv.spec_sample_workspace(mode, logits)),
        "lmhead": (lambda s: sv.spec_lmhead_sample(mode, hidden, weight, tok, acc, draft_tokens=drafts, stream=s),
                   sv.spec_lmhead_sample_workspace(mode, hidden, weight)),
        "commit": (lambda s: [sv.spec_commit(sv.SPEC_COMMIT_CHAIN, lens, none, 1, stream=s)[:4]], 256),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["verify", "window", "sample", "lmhead", "commit"])
def test_round_calls_and_a_dropped_tensor_still_being_read(sv, name, raw):
    torch = torch_mod()
    call, need = round_calls(sv)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temp = torch.full((need,), 3, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    seen = temp.clone()
    del temp
    got = call(side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert bool((seen == 3).all()) and all(torch.equal(a, b) for a, b in zip(got, want))
