"""Views whose dimensions of one element have strides that no vector access could use (one token, one kv head,
one page, pages of one token) give what contiguous tensors give, bit for bit."""

import pytest

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def odd(x):
    """x's values in a tensor that is as far from aligned as its shape allows."""
    torch = torch_mod()
    strides, at = [], 1
    for i, n in enumerate(reversed(x.shape)):
        strides.insert(0, at if n > 1 or i == 0 else 3 * at + 1)
        at *= n
    out = torch.empty_strided(x.shape, strides, dtype=x.dtype, device=x.device)
    return out.copy_(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,ctx,Hq,Hkv,pages,page", [(1, 200, 8, 2, 13, 16), (1, 200, 32, 1, 4, 64), (1, 100, 4, 1, 1, 128),
                                                     (40, 300, 2, 1, 5, 64), (1, 9, 8, 1, 9, 1), (50, 256, 4, 1, 1, 256),
                                                     (40, 300, 1, 1, 3, 128)])
def test_paged(sv, T, ctx, Hq, Hkv, pages, page, dtype):
    torch = torch_mod()
    g = torch.Generator().manual_seed(ctx + T)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    norm = lambda *s: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, kn, vn = norm(T, Hq, 64), norm(T, Hkv, 64), norm(T, Hkv, 64)
    k, v = norm(pages, Hkv, page, 64), norm(pages, Hkv, page, 64)
    table, start, lens = torch.randperm(pages, generator=g).to(torch.int32).cuda()[None], i32([0, T]), i32([ctx])
    got = []
    for f in (lambda x: x.clone(), odd):
        kk, vv, o = f(k), f(v), f(torch.zeros(T, Hq, 64, device="cuda"))
        # strides of k_new and v_new may differ where they do not matter
        sv.spec_paged_attn(f(q), kk, vv, f(table), start, lens, o, max_q=T, k_new=f(kn),
                           v_new=vn if T == 1 or Hkv == 1 else f(vn))
        got.append((o, kk, vv))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got)) and bool(torch.isfinite(got[0][0]).all())
    assert float(got[0][0].abs().sum()) > 0 and not torch.equal(got[0][1], k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (1, 1, 1), (300, 4, 1)])
def test_prefill(sv, T, Hq, Hkv, dtype):
    torch = torch_mod()
    g = torch.Generator().manual_seed(T)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = (torch.randn(T, h, 64, generator=g).to(t).cuda() for h in (Hq, Hkv, Hkv))
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    a = sv.spec_prefill_attn(q, k, v, start, torch.zeros(T, Hq, 64, device="cuda"))
    b = sv.spec_prefill_attn(odd(q), odd(k), v, start, odd(torch.zeros(T, Hq, 64, device="cuda")))
    assert torch.equal(a, b) and bool(torch.isfinite(a).all())
