"""What follows spec_paged_attn in a stream or a captured graph sees all that the call writes, also where no
segment is cut over CTAs and the call's second kernel has nothing to join: contexts of up to 128 keys under a
table with room for 1024, the first tokens of every generation."""

import numpy as np
import pytest

from oracle import serve as os_

from .helpers import torch_mod

pytestmark = pytest.mark.gpu

SENTINEL = 7.5


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


@pytest.mark.parametrize("B,n,Hq,Hkv,D", [(1, 1, 32, 8, 128), (8, 1, 32, 8, 128), (16, 4, 32, 8, 64), (40, 1, 4, 1, 128),
                                          (3, 8, 4, 1, 128)])
def test_whole_segments_and_what_follows(sv, B, n, Hq, Hkv, D):
    torch = torch_mod()
    g = torch.Generator().manual_seed(B + n)
    page, cols = 16, 64
    norm = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    kv_len = torch.randint(n, 129, (B,), generator=g, dtype=torch.int32)
    q, kn, vn = norm(B * n, Hq, D), norm(B * n, Hkv, D), norm(B * n, Hkv, D)
    k0, v0 = norm(B * 8, Hkv, page, D), norm(B * 8, Hkv, page, D)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    table[:, :8] = torch.randperm(B * 8, generator=g).view(B, 8).to(torch.int32)
    table, lens = table.cuda(), kv_len.cuda()
    start = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    k, v = k0.clone(), v0.clone()
    o = torch.empty((B * n, Hq, D), dtype=torch.bfloat16, device="cuda")
    # consumers: copies of all that the call writes, and a draft window over the first token's output, whose
    # kernel is itself a programmatic dependent of the call's last one
    o_seen, k_seen, v_seen = torch.empty_like(o), torch.empty_like(k), torch.empty_like(v)
    ring_k, ring_v, pos = norm(B, Hkv, 64, D), norm(B, Hkv, 64, D), torch.full((B,), 64, dtype=torch.int32, device="cuda")
    w_seen = torch.empty((B, Hq, D), device="cuda")
    ws = torch.empty(sv.spec_paged_attn_workspace(q, k, table, o, max_q=n), dtype=torch.uint8, device="cuda")
    wws = torch.empty(sv.spec_draft_window_attn_workspace(o.view(B, n, Hq, D)[:, 0], ring_k, w_seen), dtype=torch.uint8,
                      device="cuda")

    def call():
        sv.spec_paged_attn(q, k, v, table, start, lens, o, max_q=n, k_new=kn, v_new=vn, workspace=ws)

    def reset():
        o.fill_(SENTINEL)
        k.copy_(k0)
        v.copy_(v0)

    def window():
        sv.spec_draft_window_attn(o.view(B, n, Hq, D)[:, 0], ring_k, ring_v, pos, w_seen, workspace=wws)

    reset()
    call()
    torch.cuda.synchronize()
    want_o, want_k, want_v = o.clone(), k.clone(), v.clone()
    window()
    torch.cuda.synchronize()
    want_w = w_seen.clone()
    f64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    ref_k, ref_v = os_.append_pages(f64(k0), f64(v0), table.cpu().numpy(), start.cpu().numpy(), kv_len.numpy(), f64(kn),
                                    f64(vn))
    assert np.array_equal(f64(want_k), ref_k) and np.array_equal(f64(want_v), ref_v)
    ref, A, S = os_.paged_attn(f64(q), ref_k, ref_v, table.cpu().numpy(), start.cpu().numpy(), kv_len.numpy())
    # P rounded to bf16 (2^-8 of sum p|v|), scores of D-term fp32 sums, the output rounded to bf16
    tol = (2.0 ** -8 + 2 * ((D + 8) * 2.0 ** -24 * S + 2.0 ** -20) + 2 * 128 * 2.0 ** -24) * A + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(f64(want_o) - ref) <= tol)

    def copies():
        o_seen.copy_(o)
        k_seen.copy_(k)
        v_seen.copy_(v)

    def check():
        torch.cuda.synchronize()
        assert torch.equal(w_seen, want_w) and torch.equal(o_seen, want_o)
        assert torch.equal(k_seen, want_k) and torch.equal(v_seen, want_v)
        assert sv.read_status(ws) == 0 and sv.read_status(wws) == 0

    for order in ((window, copies), (copies, window)):
        for _ in range(5):
            reset()
            call()
            for f in order:
                f()
            check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            reset()
            call()
            for f in order:
                f()
        for _ in range(20):
            w_seen.fill_(SENTINEL)
            graph.replay()
            check()
