"""Random calls of the serving operators against 64 bits, with seeds of their own: ragged batches with resting
sequences and lengths that are too short, odd page sizes, tables far wider than the contexts, windows, strided
outputs, NaN in every slot past a sequence's end; each call repeated bit for bit on another stream, with the
binding's own workspace and beside a call on the current one.

SPEC_RANDOM_CALLS sets how many calls each test makes (30 by default), SPEC_RANDOM_SEED where the seeds begin."""

import math
import os
import random

import pytest

from .helpers import torch_mod

pytestmark = pytest.mark.gpu

CALLS = int(os.environ.get("SPEC_RANDOM_CALLS", "30"))
SEED = int(os.environ.get("SPEC_RANDOM_SEED", "0"))
SENTINEL = 7.5


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


def log_uniform(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))


def draw(rng, paged):
    """Sizes of one attention call that 64 bits can check in a moment."""
    while True:
        Hkv, G, D = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 32]), rng.choice([64, 128])
        B = rng.choice([1, 1, 2, 3, 5, 10, 33, 64, 65, 100, 300])
        top = rng.choice([1, 8, 64, 600, 2000])
        q = [log_uniform(rng, 1, top) if rng.random() > 0.1 else 0 for _ in range(B)]
        if rng.random() < 0.3:
            q = [n if rng.random() < 0.1 else 1 for n in q]
        q[0] = q[0] or 1
        far = rng.choice([10, 100, 300, 3000, 30000])
        kv = [n + (log_uniform(rng, 1, far) - 1 if rng.random() < 0.6 else rng.randint(0, 40)) for n in q]
        if not paged:
            kv = list(q)
        if sum(a * b for a, b in zip(q, kv)) * Hkv * G * D > 4e9 or sum(kv) * Hkv * D > 6e7 or sum(q) * Hkv * G * D > 3e7:
            continue
        if paged and rng.random() < 0.15:
            b = rng.randrange(B)
            kv[b] = max(0, q[b] - 1 - rng.randint(0, 3))
        return dict(q=q, kv=kv, Hkv=Hkv, G=G, D=D, B=B, window=rng.choice([0, 0, 0, 1, 5, 64, 127, 128, 200, 1000, 2 ** 31 - 1,
                                                                          2 ** 40]))


def reference(c, q, K, V, window, dtype, o_dtype, L):
    """o of one sequence in 64 bits and the bound of an element's error (see test_gpu_serve_attn)."""
    torch = torch_mod()
    n, Hkv, G, D = q.shape[0], c["Hkv"], c["G"], c["D"]
    x = q.double().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
    K, V = K.double(), V.double()
    scale = 1 / math.sqrt(D)
    pos, key = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
    seen = (key <= pos) & ((key > pos - window) if window else (key >= 0))
    s = (x @ K.transpose(1, 2) * scale).view(Hkv, G, n, L).masked_fill(~seen, -math.inf)
    p = torch.softmax(s, -1).view(Hkv, G * n, L)
    back = lambda y: y.view(Hkv, G, n, D).permute(2, 0, 1, 3).reshape(n, Hkv * G, D)  # noqa: E731
    ref, A = back(p @ V), back(p @ V.abs())
    S = float((x.abs() @ K.abs().transpose(1, 2)).max()) * scale
    r = (D + 8) * 2.0 ** -24 * S + 2.0 ** -20
    tol = (2 * r + 2 * L * 2.0 ** -24) * A + (2.0 ** -8 * A if dtype is torch.bfloat16 else 0)
    return ref, tol + (2.0 ** -8 if o_dtype is torch.bfloat16 else 2.0 ** -24) * ref.abs() + 1e-30


@pytest.mark.parametrize("kind", ["paged", "paged-append", "prompt"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention(sv, kind, dtype):
    torch = torch_mod()
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    side = torch.cuda.Stream()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for call_no in range(CALLS):
        seed = SEED + call_no
        rng = random.Random(f"{kind}/{dtype}/{seed}")
        g = torch.Generator(device="cuda").manual_seed(rng.randrange(2 ** 40))
        norm = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
        c = draw(rng, kind != "prompt")
        q_len, kv, Hkv, D, B, window = c["q"], c["kv"], c["Hkv"], c["D"], c["B"], c["window"]
        Hq, lead = Hkv * c["G"], rng.randint(0, 3)
        start = [lead + sum(q_len[:b]) for b in range(B + 1)]
        T, o_dtype = start[-1] + rng.randint(0, 3), rng.choice([t, torch.float32])
        q = norm(T, Hq, D)
        q[:lead], q[start[-1]:] = float("nan"), float("nan")
        pad = rng.choice([0, 0, 1, 8])

        def new_o():
            return torch.full((T, Hq, D + pad), SENTINEL, dtype=o_dtype, device="cuda")[:, :, pad:]

        d_start, d_len = i32(start), i32(kv)
        bad = [n > 0 and length < n for n, length in zip(q_len, kv)]
        what = f"{kind} {dtype} seed {seed}: {c}"
        if kind == "prompt":
            k, v = norm(T, Hkv, D), norm(T, Hkv, D)
            for x in (k, v):
                x[:lead], x[start[-1]:] = float("nan"), float("nan")
            keys = [(k[a:e].transpose(0, 1), v[a:e].transpose(0, 1)) for a, e in zip(start, start[1:])]
            need = sv.spec_prefill_attn_workspace(q, k, d_start, q)
            call = lambda o, **kw: sv.spec_prefill_attn(q, k, v, d_start, o, window=window, **kw)  # noqa: E731
        else:
            page = rng.choice([1, 2, 8, 16, 16, 17, 24, 32, 48, 64, 100, 128, 256])
            per = [-(-n // page) for n in kv]
            pages = sum(per) + 2
            k, v = norm(pages, Hkv, page, D), norm(pages, Hkv, page, D)
            if rng.random() < 0.3:  # token-major pages
                k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
            order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
            table = torch.full((B, max(*per, 1) + rng.choice([0, 0, 3, 2000 // page + 1])), -1, dtype=torch.int32,
                               device="cuda")
            at = 0
            for b in range(B):
                table[b, :per[b]] = order[at:at + per[b]]
                at += per[b]
                if kv[b] % page:
                    last = int(table[b, per[b] - 1])
                    k[last, :, kv[b] % page:], v[last, :, kv[b] % page:] = float("nan"), float("nan")
            kw_new = {}
            if kind == "paged-append":
                kw_new = dict(k_new=norm(T, Hkv, D), v_new=norm(T, Hkv, D))
            keys = []
            for b in range(B):
                idx = table[b, :per[b]].long()
                pair = [x[idx].transpose(0, 1).reshape(Hkv, -1, D)[:, :kv[b]].clone() for x in (k, v)]
                if kw_new and not bad[b]:
                    for x, name in zip(pair, ("k_new", "v_new")):
                        x[:, kv[b] - q_len[b]:] = kw_new[name][start[b]:start[b + 1]].transpose(0, 1)
                keys.append(pair)
            max_q = max(q_len) + rng.choice([0, 0, 0, 5, 10 ** 6])
            need = sv.spec_paged_attn_workspace(q, k, table, q, max_q=max_q)
            call = lambda o, **kw: sv.spec_paged_attn(q, k, v, table, d_start, d_len, o, max_q=max_q,  # noqa: E731
                                                      window=window, **kw_new, **kw)
        o, again, beside = new_o(), new_o(), new_o()
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        call(o, workspace=ws)
        torch.cuda.synchronize()
        assert sv.read_status(ws) == (sv.binding.SPEC_STATUS_BAD_KV_LEN if any(bad) else 0), what
        call(beside)
        if kind != "paged-append":  # two calls that append to the same slots must not overlap
            call(again, stream=side)
        else:
            torch.cuda.synchronize()
            call(again, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o, again) and torch.equal(o, beside), what
        assert bool((o[:lead] == SENTINEL).all()) and bool((o[start[-1]:] == SENTINEL).all()), what
        for b in range(B):
            if q_len[b] == 0:
                continue
            got = o[start[b]:start[b + 1]].double()
            if bad[b]:
                assert bool((got == 0).all()), what
                continue
            ref, tol = reference(c, q[start[b]:start[b + 1]], *keys[b], window, t, o_dtype, kv[b])
            over = float(((got - ref).abs() / tol).max())
            assert over <= 1, f"{over} times the bound in sequence {b}, {what}"
        if kind == "paged-append":
            for b in range(B):
                if q_len[b] and not bad[b]:
                    idx = table[b, :per[b]].long()
                    for x, y in zip((k, v), keys[b]):
                        assert torch.equal(x[idx].transpose(0, 1).reshape(Hkv, -1, D)[:, :kv[b]], y), what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs(sv, dtype):
    torch = torch_mod()
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    side = torch.cuda.Stream()
    for call_no in range(2 * CALLS):
        seed = SEED + call_no
        rng = random.Random(f"logprobs/{dtype}/{seed}")
        g = torch.Generator(device="cuda").manual_seed(rng.randrange(2 ** 40))
        N = rng.choice([1, 2, 3, 7, 40, 152, 153, 607, 608, 2000])
        V = rng.choice([1, 2, 7, 31, 32, 33, 255, 1000, 1024, 4097, 32000, 50257, 128256, rng.randint(1, 200000)])
        V = min(V, 40_000_000 // N)
        K, pad = min(rng.choice([0, 1, 2, 5, 16, 20, 31, 32]), V), rng.choice([0, 0, 1, 3, 8, 64])
        kind = rng.choice(["normal", "ties", "rising", "falling", "masked", "one", "large", "nothing"])
        x = torch.randn(N, V, generator=g, device="cuda") * 3
        if kind == "ties":
            x = x.round()
        elif kind == "rising":
            x = torch.linspace(-50, 50, V, device="cuda").expand(N, V).clone()
        elif kind == "falling":
            x = torch.linspace(50, -50, V, device="cuda").expand(N, V).clone()
        elif kind == "masked":
            x = x.masked_fill(torch.rand(N, V, generator=g, device="cuda") < rng.choice([0.3, 0.99]), -math.inf)
        elif kind == "large":
            x = x * 1e4
        elif kind == "one":
            x = torch.full((N, V), -math.inf, device="cuda")
            x[torch.arange(N), torch.randint(0, V, (N,))] = 3.0
        elif kind == "nothing":
            x[::3] = -math.inf
        base = torch.full((N, V + pad), float("nan"), dtype=t, device="cuda")
        at = rng.randint(0, pad)
        logits = base[:, at:at + V]
        logits.copy_(x)
        tok = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        what = f"logprobs {dtype} seed {seed}: N {N} V {V} K {K} pad {pad} {kind}"

        def outputs():
            return dict(logprobs=torch.full((N,), 9.0, device="cuda"), entropy=torch.full((N,), 9.0, device="cuda"),
                        **(dict(top_ids=torch.full((N, K), -9, dtype=torch.int32, device="cuda"),
                                top_logprobs=torch.full((N, K), 9.0, device="cuda")) if K else {}))
        outs = [outputs() for _ in range(3)]
        torch.cuda.synchronize()
        sv.spec_token_logprobs(logits, tok, **outs[0])
        sv.spec_token_logprobs(logits, tok, stream=side, **outs[1])
        sv.spec_token_logprobs(logits, tok, **outs[2])
        torch.cuda.synchronize()
        for other in outs[1:]:
            assert all(torch.equal(outs[0][n], other[n]) for n in other), what
        # bounds as in test_gpu_logprobs_rows, for a row in one CTA (slices add less)
        E = 32 if dtype == "bf16" else 16
        log_v = math.log(V) if V > 1 else 0.0
        r = (E / 2 + 2) * 2.0 ** -24 + (-(-V // (128 * E)) + 32) * (2.0 ** -22 + 3 * 2.0 ** -24) + 2.0 ** -22 + 2.0 ** -23 * log_v
        z = logits.double()
        m = z.max(1, keepdim=True).values
        live = torch.isfinite(m[:, 0])
        d = z - m
        ref = torch.where(live[:, None], d - d.exp().sum(1, keepdim=True).log(), -math.inf)

        def near(got, at_ids, name):
            want, dist = ref.gather(1, at_ids), d.gather(1, at_ids).abs()
            fin = torch.isfinite(want)
            got = got.double()
            assert torch.equal(got[~fin], want[~fin]), f"{name} {what}"
            assert bool(((got - want).abs() <= r + 2.0 ** -23 * (dist + log_v))[fin].all()), f"{name} {what}"
        near(outs[0]["logprobs"][:, None], tok.long()[:, None], "logprobs")
        p = ref.exp()
        H = -torch.where(p > 0, p * ref, 0.0).sum(1)
        err = (outs[0]["entropy"].double() - H).abs()
        assert float(err.max()) <= r + 2 * r * log_v + 2.0 ** -22 * log_v + 1e-30, f"entropy {what}"
        if K:
            order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :K]
            assert torch.equal(outs[0]["top_ids"].long(), order), what
            near(outs[0]["top_logprobs"], order, "top")
