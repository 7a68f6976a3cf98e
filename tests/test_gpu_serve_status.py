"""The status word of calls that a captured graph replays: a replay on bad data flags it, the next one on good
data is clean, and a replay of another graph that shares the workspace changes nothing about that."""

import pytest

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def paged_setup(sv, q_len, cols, append, dtype, window=0):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(1)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    norm = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    B, T, page = len(q_len), sum(q_len), 16
    q, k, v = norm(T, 4, 64), norm(B * 20, 2, page, 64), norm(B * 20, 2, page, 64)
    new = dict(k_new=norm(T, 2, 64), v_new=norm(T, 2, 64)) if append else {}
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    table[:, :20] = torch.arange(B * 20, dtype=torch.int32, device="cuda").view(B, 20)
    start, lens = i32([sum(q_len[:b]) for b in range(B + 1)]), i32([300] * B)
    o = torch.empty((T, 4, 64), device="cuda")
    ws = torch.empty(sv.spec_paged_attn_workspace(q, k, table, o, max_q=max(q_len)), dtype=torch.uint8, device="cuda")

    def call():
        sv.spec_paged_attn(q, k, v, table, start, lens, o, max_q=max(q_len), window=window, workspace=ws, **new)
    good = lens.clone(), table.clone(), start.clone()

    def spoil(kind):
        lens.copy_(good[0])
        table.copy_(good[1])
        start.copy_(good[2])
        if kind == sv.binding.SPEC_STATUS_BAD_KV_LEN:
            lens[1] = -1
        elif kind == sv.SPEC_STATUS_BAD_PAGE:
            table[1, 17] = -7
        elif kind == sv.SPEC_STATUS_BAD_RANGE:
            start[B] = T + 1
    return call, spoil, o, ws


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("q_len,cols,window", [([2, 1, 3], 20, 0), ([2, 1, 3], 300, 0), ([40, 30, 60], 20, 0),
                                               ([40, 30, 60], 300, 0), ([40, 30, 60], 300, 64)])
def test_paged(sv, q_len, cols, window, append, dtype):
    torch = torch_mod()
    call, spoil, o, ws = paged_setup(sv, q_len, cols, append, dtype, window)
    call()
    torch.cuda.synchronize()
    want = o.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    kinds = [0, sv.binding.SPEC_STATUS_BAD_KV_LEN, 0, sv.SPEC_STATUS_BAD_PAGE, sv.SPEC_STATUS_BAD_RANGE, 0]
    for turn in range(3):
        for i, kind in enumerate(kinds):
            spoil(kind)
            graphs[(turn + i) % 2].replay()
            torch.cuda.synchronize()
            assert sv.read_status(ws) == kind
            if kind == 0:
                assert torch.equal(o, want)
            # a call outside the graphs in between
            call()
            torch.cuda.synchronize()
            assert sv.read_status(ws) == kind


@pytest.mark.parametrize("N,V", [(3, 50257), (700, 5000)])
def test_logprobs(sv, N, V):
    torch = torch_mod()
    x = torch.randn(N, V, device="cuda")
    tok = torch.zeros(N, dtype=torch.int32, device="cuda")
    lp = torch.empty(N, device="cuda")
    ws = torch.empty(sv.spec_token_logprobs_workspace(x, 0), dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            sv.spec_token_logprobs(x, tok, lp, workspace=ws)
    for i in range(8):
        bad = i % 3 == 1
        tok[N - 1] = V if bad else 0
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert sv.read_status(ws) == (sv.binding.SPEC_STATUS_BAD_TOKEN if bad else 0)
