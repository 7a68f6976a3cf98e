"""GPU parity of spec_token_logprobs against the float64 oracle, and a serving round over all operators.

Bounds, derived: x - max is rounded once (2^-24 relative); 2^x is off by 2^-22 relative plus 2^-24 |d| log2(e)
for the rounded exponent, whose weighted mean is at most 2^-24 * 1.5 * H'; a thread adds about V / 256 + 16 terms
in fp32 and the joins 64 more, so s is off by r = (V / 256 + 80) 2^-24 + 2^-21 relatively, and log s by as
much absolutely.  logprob: r + 2^-23 (|x - max| + |log s|).  Entropy: log s - w / s with w = sum |d| e of the
same relative error: r (1 + 2 w / s) + 2^-22 (log s + w / s).
"""

import numpy as np
import pytest

from oracle import serve as os_

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def run(sv, x, tok, K, entropy=True, stream=None):
    torch = torch_mod()
    N = x.shape[0]
    lp = torch.full((N,), 9.0, device="cuda")
    ent = torch.full((N,), 9.0, device="cuda") if entropy else None
    ids = torch.full((N, K), -9, dtype=torch.int32, device="cuda") if K else None
    top = torch.full((N, K), 9.0, device="cuda") if K else None
    ws = torch.full((sv.spec_token_logprobs_workspace(x, K),), 255, dtype=torch.uint8, device="cuda")
    sv.spec_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=top, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return lp, ent, ids, top, sv.read_status(ws)


def verify(sv, x, tok, K):
    """x: a device tensor; compares every output with the oracle on the stored values."""
    lp, ent, ids, top, st = run(sv, x, tok, K)
    xs = x.double().cpu().numpy()
    V = xs.shape[1]
    rl, re, ri, rt = os_.token_logprobs(xs, tok.cpu().numpy(), K)
    with np.errstate(invalid="ignore"):
        spread = np.nan_to_num(xs.max(1) - np.where(np.isfinite(xs), xs, np.inf).min(1), posinf=0, neginf=0)
    r = (V / 256 + 80) * 2.0 ** -24 + 2.0 ** -21
    logs = np.log(V)
    tol = r + 2.0 ** -23 * (spread + logs)
    for got, ref, t in ((lp, rl, tol), *(((top[:, i], rt[:, i], tol)) for i in range(K))):
        got = got.double().cpu().numpy()
        fin = np.isfinite(ref)
        assert np.array_equal(got[~fin], ref[~fin])
        assert np.all(np.abs(got[fin] - ref[fin]) <= t[fin])
    e = ent.double().cpu().numpy()
    assert np.all(np.abs(e - re) <= r * (1 + 2 * logs) + 2.0 ** -22 * 2 * logs + 1e-30 + 2 * r)
    if K:
        assert np.array_equal(ids.cpu().numpy(), ri)
    return st


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (1, 2, 2), (3, 5, 0), (2, 33, 32), (5, 1000, 5), (1, 128256, 20),
                                   (7, 50257, 32), (400, 1001, 3), (320, 32000, 5), (2, 40000, 1)])
def test_parity(sv, N, V, K, dtype):
    torch = torch_mod()
    g = torch.Generator().manual_seed(N + V)
    x = (torch.randn(N, V, generator=g) * 2).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    assert verify(sv, x, tok, K) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(2, 300), (2, 20000), (330, 5000)])
def test_ties_masks_and_bad_tokens(sv, N, V, dtype):
    """Few distinct values (ties to the lower id across vectors, warps, slices), -0 against +0, masked
    ids, rows with fewer ids than alternatives, rows of nothing, tokens outside the vocabulary."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(V)
    x = torch.randint(-2, 3, (N, V), generator=g).float()
    x[0] = 0.0
    x[0, ::3] = -0.0
    x[1, 7:] = -float("inf")
    if N > 2:
        x[2] = -float("inf")
        x[3] = -float("inf")
        x[3, V - 2] = 1.5
        x[4, V // 2:] = -float("inf")
        x[5] = torch.arange(V).float() / V * 8  # ascending: every batch beats the last
        x[6] = -torch.arange(V).float() / V * 8
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    tok[0] = V
    if N > 2:
        tok[7], tok[8] = -1, 2 ** 31 - 1
    st = verify(sv, x, tok.cuda(), 32)
    assert st == sv.SPEC_STATUS_BAD_TOKEN
    assert verify(sv, x, torch.zeros(N, dtype=torch.int32, device="cuda"), 5) == 0


def test_strided_unaligned_rows_and_optional_outputs(sv):
    torch = torch_mod()
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(6, 5003, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
        base[:, 0] = float("nan")
        base[:, -2:] = float("inf")
        x = base[:, 1:5001]
        tok = torch.tensor([0, 4999, 17, 2500, 1, 3], dtype=torch.int32, device="cuda")
        assert verify(sv, x, tok, 7) == 0
        lp, _, _, _, st = run(sv, x, tok, 0, entropy=False)
        full = run(sv, x, tok, 7)
        assert st == 0 and bool((lp == full[0]).all())
        only = torch.empty(6, device="cuda")
        sv.spec_token_logprobs(x, None, None, entropy=only)
        assert bool((only == full[1]).all())


def test_far_rows_and_large_logits(sv):
    """Row offsets past 2^31 elements, and logits whose exponentials would overflow."""
    torch = torch_mod()
    V, N = 50000, 43000  # 2.15e9 elements
    x = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(9)
    x[-1] = (torch.randn(V, generator=g) * 300).to(torch.bfloat16).cuda()
    tok = torch.full((N,), 3, dtype=torch.int32, device="cuda")
    lp, ent, ids, top, st = run(sv, x, tok, 2)
    assert st == 0
    rl, re, ri, rt = os_.token_logprobs(x[-1:].double().cpu().numpy(), np.array([3]), 2)
    assert abs(float(lp[-1]) - rl[0]) <= 2.0 ** -22 * abs(rl[0]) + 1e-4 and abs(float(ent[-1]) - re[0]) < 1e-4
    assert ids[-1].tolist() == list(ri[0]) and ids[0].tolist() == [0, 1]
    assert float((lp[:-1] + np.log(V)).abs().max()) < 1e-4 and float((ent[:-1] - np.log(V)).abs().max()) < 2e-4


@pytest.mark.parametrize("N", [3, 700])
def test_graph_and_streams(sv, N):
    torch = torch_mod()
    xs = [torch.randn(N, 20001, device="cuda") for _ in range(2)]
    tok = torch.randint(0, 20001, (N,), dtype=torch.int32, device="cuda")
    want = [run(sv, x, tok, 4) for x in xs]
    x, lp = xs[0].clone(), torch.empty(N, device="cuda")
    ids, top = torch.empty((N, 4), dtype=torch.int32, device="cuda"), torch.empty((N, 4), device="cuda")
    ws = torch.empty(sv.spec_token_logprobs_workspace(x, 4), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_token_logprobs(x, tok, lp, top_ids=ids, top_logprobs=top, workspace=ws)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert bool((lp == want[i][0]).all()) and bool((ids == want[i][2]).all()) and bool((top == want[i][3]).all())
    s = torch.cuda.Stream()
    for i in (0, 1):
        got = run(sv, xs[i], tok, 4, stream=s)
        assert all(bool((a == b).all()) for a, b in zip(got[:4], want[i][:4]))


def test_a_serving_round(sv):
    """Prompts through spec_prefill_attn and, chunk by chunk, through spec_paged_attn's append (the same
    answer), then a draft chain verified over the pages, committed, and its tokens scored."""
    torch = torch_mod()
    g = torch.Generator().manual_seed(11)
    B, Hq, Hkv, D, page, V, gamma = 2, 8, 2, 64, 16, 1500, 4
    lens = [150, 61]
    T = sum(lens)
    norm = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = norm(T, Hq, D), norm(T, Hkv, D), norm(T, Hkv, D)
    whole = sv.spec_prefill_attn(q, k, v, i32([0, 150, 211]), torch.empty((T, Hq, D), device="cuda"))
    kp = torch.full((40, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.randperm(40, generator=g)[:24].view(2, 12).to(torch.int32).cuda()
    done = [0, 0]
    parts = [torch.empty(n, Hq, D, device="cuda") for n in lens]
    for sizes in ((70, 60), (79, 0), (1, 1)):
        rows = [slice(sum(lens[:b]) + done[b], sum(lens[:b]) + done[b] + sizes[b]) for b in range(B)]
        cat = lambda x: torch.cat([x[r] for r in rows])  # noqa: E731
        o = torch.empty((sum(sizes), Hq, D), device="cuda")
        lens_now = [done[b] + sizes[b] for b in range(B)]
        sv.spec_paged_attn(cat(q), kp, vp, table, i32([0, sizes[0], sum(sizes)]), i32(lens_now), o, max_q=max(sizes),
                           k_new=cat(k), v_new=cat(v))
        for b in range(B):
            parts[b][done[b]:lens_now[b]] = o[sum(sizes[:b]):sum(sizes[:b + 1])]
        done = lens_now
    # both round P to bf16 against their own running maxima: 2^-8 of sum p|v| each
    assert float((torch.cat(parts) - whole).abs().max()) <= 2 * 2.0 ** -8 * float(v.abs().max())

    n = gamma + 1
    kv_len = i32([x + n for x in lens])
    qn, kn, vn = norm(B * n, Hq, D), norm(B * n, Hkv, D), norm(B * n, Hkv, D)
    start = i32([0, n, 2 * n])
    o = torch.empty((B * n, Hq, D), device="cuda")
    sv.spec_paged_attn(qn, kp, vp, table, start, kv_len, o, max_q=n, k_new=kn, v_new=vn)
    ref, A, S = os_.paged_attn(*(x.double().cpu().numpy() for x in (qn, kp, vp)), table.cpu().numpy(),
                               start.cpu().numpy(), kv_len.cpu().numpy())
    err = np.abs(o.double().cpu().numpy() - ref)
    assert np.all(err <= (2.0 ** -8 + 2.0 ** -12) * A + 1e-6)
    logits = torch.randn(B, n, V, generator=g).cuda()
    drafts = logits.argmax(-1)[:, :gamma].to(torch.int32)
    drafts[1, 2] = (drafts[1, 2] + 1) % V
    out, acc = torch.empty((B, n), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    sv.spec_sample(sv.SPEC_SAMPLE_CHAIN_GREEDY, logits, out, acc, draft_tokens=drafts)
    sv.spec_commit(sv.SPEC_COMMIT_CHAIN, kv_len, acc, n)
    assert acc.tolist() == [4, 2] and kv_len.tolist() == [lens[0] + 5, lens[1] + 3]
    rows = logits.view(B * n, V)
    lp = torch.empty(B * n, device="cuda")
    ids, top = torch.empty((B * n, 1), dtype=torch.int32, device="cuda"), torch.empty((B * n, 1), device="cuda")
    sv.spec_token_logprobs(rows, out.view(-1), lp, top_ids=ids, top_logprobs=top)
    want = torch.log_softmax(rows.double(), -1)
    emitted = out.view(-1) >= 0
    got = want.gather(1, out.view(-1).clamp(min=0).long()[:, None])[:, 0]
    assert float((lp.double() - got)[emitted].abs().max()) < 1e-5
    assert bool((ids.view(B, n)[out >= 0] == out[out >= 0]).all())  # greedy tokens are the top alternatives
    assert float((top[:, 0].double() - want.max(-1).values).abs().max()) < 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks_of_the_lowest_value(sv, dtype):
    """Ids masked by the type's lowest finite value take no part; a row of nothing else is uniform."""
    torch = torch_mod()
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    low = torch.finfo(t).min
    V = 9001
    x = (torch.randn(3, V, generator=torch.Generator().manual_seed(1)) * 3).to(t)
    x[:2, 100:] = low
    x[1, :100] = low
    ref = x.clone()
    ref[0, 100:] = -float("inf")
    tok = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    got, want = run(sv, x.cuda(), tok, 32), run(sv, ref.cuda(), tok, 32)
    for a, b in zip(got[:4], want[:4]):
        assert bool((a[0] == b[0]).all()) and bool((a[2] == b[2]).all())
    # log V by a fp32 sum of V ones and logf: half an ulp of log V, twice
    assert abs(float(got[0][1]) + np.log(V)) < 2e-6 and abs(float(got[1][1]) - np.log(V)) < 2e-6
    assert got[2][1].tolist() == list(range(32))
