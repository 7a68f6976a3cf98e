"""spec_token_logprobs where a row is one CTA's (608 rows and more), at large vocabularies, against 64 bits.

Bounds, derived from the kernel's sums.  A thread of an unsliced row adds its elements in batches of E = 32
(bf16) or 16 (fp32), each batch as two chains of E / 2 terms, and carries the sum over nb batches, nb = V / (128 E)
rounded up, each of which can rescale it (2^x off by 2^-22, and three roundings).  The joins of 32 lanes, four
warps and the row's ends are 9 steps of the same kind.  A term's own error is 2^-22 of 2^x and, from the
rounded difference and exponent, 2^-23 |d|, whose mean over the row is w / s <= log V (the entropy is not
negative).  So s is off relatively by
    r = (E / 2 + 2) 2^-24 + (nb + 9) (2^-22 + 3 2^-24) + 2^-22 + 2^-23 log V
and log s absolutely by as much, plus its own rounding.  A log probability (x - m) - log s: r + 2^-23 (|x - m| +
log V).  The entropy log s - w / s, w of twice s's relative error: r + 2 r log V + 2^-23 2 log V."""

import numpy as np
import pytest

from .helpers import torch_mod

pytestmark = pytest.mark.gpu


def bounds(V, dtype):
    E = 32 if dtype == "bf16" else 16
    nb = -(-V // (128 * E))
    log_v = np.log(V)
    r = (E / 2 + 2) * 2.0 ** -24 + (nb + 9) * (2.0 ** -22 + 3 * 2.0 ** -24) + 2.0 ** -22 + 2.0 ** -23 * log_v
    return r, r + 2 * r * log_v + 2.0 ** -22 * log_v


def values(kind, N, V, t):
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(N, V, generator=g, device="cuda") * 3
    if kind == "rising":  # every batch moves the reference
        x = x * 0.01 + torch.linspace(-20, 20, V, device="cuda")
    elif kind == "falling":
        x = x * 0.01 + torch.linspace(20, -20, V, device="cuda")
    elif kind == "flat":
        x = x * 0
    elif kind == "ties":
        x = x.round()
    return x.to(t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["normal", "rising", "falling", "flat", "ties"])
@pytest.mark.parametrize("N,V,K", [(608, 32000, 5), (640, 128256, 20), (700, 50257, 32)])
def test_unsliced_rows(N, V, K, kind, dtype):
    torch = torch_mod()
    import speculative_decoding_verify_attn_gb300 as sv
    x = values(kind, N, V, torch.bfloat16 if dtype == "bf16" else torch.float32)
    tok = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    lp, ent = torch.full((N,), 9.0, device="cuda"), torch.full((N,), 9.0, device="cuda")
    ids, top = torch.full((N, K), -9, dtype=torch.int32, device="cuda"), torch.full((N, K), 9.0, device="cuda")
    sv.spec_token_logprobs(x, tok, lp, entropy=ent, top_ids=ids, top_logprobs=top)
    tol_lp, tol_ent = bounds(V, dtype)
    log_v = np.log(V)
    for r in range(0, N, 64):  # 64 rows of 128256 in 64 bits at a time
        z = x[r:r + 64].double()
        d = z - z.max(1, keepdim=True).values
        ref = d - d.exp().sum(1, keepdim=True).log()
        order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :K]
        assert torch.equal(ids[r:r + 64].long(), order)
        t = tok[r:r + 64].long()[:, None]
        near = lambda got, at: ((got.double() - ref.gather(1, at)).abs() - tol_lp  # noqa: E731
                                - 2.0 ** -23 * (d.gather(1, at).abs() + log_v)).max()
        assert float(near(lp[r:r + 64, None], t)) <= 0 and float(near(top[r:r + 64], order)) <= 0
        H = -(ref.exp() * ref).sum(1)
        assert float((ent[r:r + 64].double() - H).abs().max()) <= tol_ent
