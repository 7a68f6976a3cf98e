"""Workloads of the serving operators around speculative decoding, for measurement.

Three operators, each with a plain form in elementary torch operations and the library's own call:

* ``paged``: attention of a ragged batch of new-token chunks over a paged KV cache
  (``spec_paged_attn``), from one token per sequence to whole prompt chunks, optionally appending
  the chunk's K/V to the pages in the same call;
* ``prompt``: causal attention over whole prompts packed one after the other
  (``spec_prefill_attn``);
* ``logprobs``: log probability of given tokens with the row's entropy and its top alternatives
  (``spec_token_logprobs``).

A case is a dict of plain values; lengths are drawn from the case alone, values from the seed.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence, one new token, a short context: the latency of a single decode step
        dict(name="paged-decode-short", op="paged", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, q_lo=1, q_hi=1,
             ctx_lo=300, ctx_hi=300, page=16, window=0, append=True),
        # a verify round of 8 sequences (gamma 4, so 5 tokens each) at 16K-32K context, K/V appended
        dict(name="paged-verify-8b", op="paged", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, q_lo=5, q_hi=5,
             ctx_lo=16384, ctx_hi=32768, page=64, window=0, append=True),
        # a verify round of 16 sequences (gamma 6) of a 64/8-head layer at 64K-128K context
        dict(name="paged-verify-70b", op="paged", dtype="bf16", B=16, Hq=64, Hkv=8, D=128, q_lo=7, q_hi=7,
             ctx_lo=65536, ctx_hi=131072, page=128, window=0, append=False),
        # continuous batching: sequences that decode, verify, rest (no token) or take a prompt chunk
        dict(name="paged-mixed", op="paged", dtype="bf16", B=24, Hq=32, Hkv=8, D=128, q_lo=0, q_hi=384,
             ctx_lo=200, ctx_hi=8192, page=16, window=0, append=True),
        # one 2048-token chunk of a long prompt
        dict(name="paged-chunk-32k", op="paged", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, q_lo=2048, q_hi=2048,
             ctx_lo=32768, ctx_hi=32768, page=64, window=0, append=False),
        # a draft model of head size 64 catching up over its 512-token window
        dict(name="paged-window-d64", op="paged", dtype="bf16", B=32, Hq=16, Hkv=4, D=64, q_lo=1, q_hi=40,
             ctx_lo=60, ctx_hi=4096, page=32, window=512, append=True),
        # fp32 cache, the small head layout
        dict(name="paged-f32", op="paged", dtype="f32", B=4, Hq=4, Hkv=1, D=64, q_lo=1, q_hi=33,
             ctx_lo=100, ctx_hi=1500, page=16, window=0, append=True),
        # a few short fp32 prompts
        dict(name="prompt-f32-short", op="prompt", dtype="f32", B=3, Hq=4, Hkv=1, D=64, q_lo=7, q_hi=400, window=0),
        # a packed batch of ragged prompts
        dict(name="prompt-packed", op="prompt", dtype="bf16", B=16, Hq=32, Hkv=8, D=128, q_lo=60, q_hi=2000,
             window=0),
        # one long prompt
        dict(name="prompt-16k", op="prompt", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, q_lo=16384, q_hi=16384,
             window=0),
        # the five verified rows of one sequence
        dict(name="logprobs-round", op="logprobs", dtype="f32", N=5, V=128256, K=5, masked=False),
        # every position of a batch of prompts, bf16 logits, a third of the ids masked out
        dict(name="logprobs-prompt", op="logprobs", dtype="bf16", N=4096, V=128256, K=20, masked=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "prompt", "logprobs"])
    if op == "logprobs":
        V = rng.choice([1000, 1024, 32000, 50257, 128256])
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), N=_log_uniform(rng, 1, 4096), V=V,
                    K=rng.choice([0, 1, 5, 20]), masked=rng.random() < 0.5)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 8])
    D = rng.choice([64, 128, 128])
    window = rng.choice([0, 0, 0, 128, 512])
    if op == "prompt":
        top = 600 if dtype == "f32" else 4096
        hi = _log_uniform(rng, 8, top)
        B = max(1, min(_log_uniform(rng, 1, 16), (1 << 29) // (hi * hi * Hkv * G)))
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, q_lo=max(1, hi // 5), q_hi=hi, window=window)
    ctx = _log_uniform(rng, 64, 8192 if dtype == "f32" else 65536)
    q_hi = min(ctx, _log_uniform(rng, 1, 64 if dtype == "f32" else 1024))
    B = max(1, min(_log_uniform(rng, 1, 32), (1 << 28) // (ctx * q_hi * Hkv * G // 4 + ctx * Hkv * D)))
    return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, q_lo=q_hi if rng.random() < 0.5 else min(1, q_hi),
                q_hi=q_hi, ctx_lo=max(q_hi, ctx // 3), ctx_hi=ctx, page=rng.choice([16, 32, 64, 128, 24]),
                window=window, append=rng.random() < 0.5)


def _lengths(case):
    """New tokens and context length (new ones included) of each sequence, from the case alone."""
    rng = random.Random("%s/%s/%s/%s" % (case["B"], case["q_lo"], case["q_hi"], case.get("ctx_hi", 0)))
    B, lo, hi = case["B"], case["q_lo"], case["q_hi"]
    if case["op"] == "prompt":
        q = [rng.randint(lo, hi) for _ in range(B)]
        return q, list(q)
    if lo == 0:  # rest, decode, verify, or a chunk of the prompt
        q = [rng.choice([0, 1, 1, 5, 5, rng.randint(16, hi), hi]) for _ in range(B)]
        q[0], q[-1] = hi, 1
    else:
        q = [rng.randint(lo, hi) for _ in range(B)]
    return q, [max(n, rng.randint(case["ctx_lo"], case["ctx_hi"])) for n in q]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        out = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")
        return out.normal_(0.0, scale, generator=g)

    s = dict(case)
    if case["op"] == "logprobs":
        N, V = case["N"], case["V"]
        s["logits"] = normal(N, V, scale=2.0)
        if case["masked"]:
            s["logits"][:, torch.randperm(V, generator=g, device="cuda")[: V // 3]] = -math.inf
        s["tokens"] = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        return s
    q_len, kv_len = _lengths(case)
    B, T, Hq, Hkv, D = case["B"], sum(q_len), case["Hq"], case["Hkv"], case["D"]
    s["max_q"], s["max_kv"] = max(q_len), max(kv_len)
    s["start"] = torch.tensor([sum(q_len[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["q"] = normal(T, Hq, D)
    if case["op"] == "prompt":
        s["k"], s["v"] = normal(T, Hkv, D), normal(T, Hkv, D)
        return s
    page = case["page"]
    per = [-(-n // page) for n in kv_len]
    pages = sum(per) + 3
    s["k_pages"], s["v_pages"] = normal(pages, Hkv, page, D), normal(pages, Hkv, page, D)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.zeros((B, max(per)), dtype=torch.int32, device="cuda")
    for b in range(B):
        s["table"][b, : per[b]] = order[sum(per[:b]): sum(per[: b + 1])]
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    if case["append"]:
        s["k_new"], s["v_new"] = normal(T, Hkv, D), normal(T, Hkv, D)
    return s


def _attend(q, k, v, q_pos, kv_end, window):
    """q [B, m, Hq, D], k and v [B, Hkv, L, D], in 32 bits; q_pos [B, m] the position of a row,
    below 0 for rows of padding; kv_end [B].  Rows see keys up to their own position, the last
    `window` of them if it is not 0."""
    B, m, Hq, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    G = Hq // Hkv
    rows = q.view(B, m, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, D)
    s = torch.matmul(rows * (1.0 / math.sqrt(D)), k.transpose(2, 3)).view(B, Hkv, G, m, L)
    key = torch.arange(L, device=q.device)
    pos = q_pos[:, :, None]
    hidden = (key > pos) | (key >= kv_end[:, None, None])
    if window:
        hidden = hidden | (key <= pos - window)
    s.masked_fill_(hidden[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp_(min=-1e30))
    s.exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, G * m, L), v).view(B, Hkv, G, m, D) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(B, m, Hq, D)


def _of_token(start, T):
    """Sequence and index in it of each packed token."""
    t = torch.arange(T, device=start.device)
    seq = torch.searchsorted(start[1:].long(), t, right=True)
    return seq, t - start.long()[seq]


def _padded(x, start, m):
    """[T, H, D] as [B, m, H, D] in 32 bits (rows past a sequence's end hold anything finite)."""
    at = start[:-1].long()[:, None] + torch.arange(m, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)].float()


def _plain_paged(s):
    start, table, page = s["start"].long(), s["table"].long(), s["page"]
    T = s["q"].shape[0]
    seq, j = _of_token(start, T)
    n = start[1:] - start[:-1]
    kv_len = s["kv_len"].long()
    if s["append"]:
        pos = kv_len[seq] - n[seq] + j
        at = table[seq, pos // page]
        s["k_pages"][at, :, pos % page] = s["k_new"]
        s["v_pages"][at, :, pos % page] = s["v_new"]

    def cache(pages):
        got = pages[table].float()  # [B, pages, Hkv, page, D]
        return got.permute(0, 2, 1, 3, 4).reshape(table.shape[0], pages.shape[1], -1, pages.shape[3])

    m = s["max_q"]
    rows = torch.arange(m, device=start.device)
    q_pos = torch.where(rows < n[:, None], (kv_len - n)[:, None] + rows, -1)
    o = _attend(_padded(s["q"], start, m), cache(s["k_pages"]), cache(s["v_pages"]), q_pos, kv_len, s["window"])
    return o[seq, j].to(s["q"].dtype)


def _plain_prompt(s):
    start = s["start"].long()
    m = s["max_q"]
    n = start[1:] - start[:-1]
    rows = torch.arange(m, device=start.device)
    q_pos = torch.where(rows < n[:, None], rows, -1)
    k, v = (_padded(s[x], start, m).transpose(1, 2) for x in ("k", "v"))
    o = _attend(_padded(s["q"], start, m), k, v, q_pos, n, s["window"])
    seq, j = _of_token(start, s["q"].shape[0])
    return o[seq, j].to(s["q"].dtype)


def _plain_logprobs(s):
    x = s["logits"].float()
    V, K = x.shape[1], s["K"]
    top = x.amax(1, keepdim=True)
    d = x - top
    e = d.exp()
    total = e.sum(1, dtype=torch.float64)
    lse = total.log()
    entropy = lse - (torch.where(e > 0, d, 0.0) * e).sum(1, dtype=torch.float64) / total
    given = d.gather(1, s["tokens"].long()[:, None])[:, 0].double() - lse
    out = {"logprobs": given.float(), "entropy": entropy.float()}
    if K:
        # the order of the floats as whole numbers (-0 as 0), the lower id first among equals
        bits = (x + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
        key = (bits << 32) + (V - 1 - torch.arange(V, device=x.device))
        key = key.topk(K, dim=1).values
        ids = V - 1 - (key & 0xFFFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = (d.gather(1, ids).double() - lse[:, None]).float()
    return out


def run(s):
    op = s["op"]
    if not own:
        if op == "logprobs":
            return _plain_logprobs(s)
        o = _plain_paged(s) if op == "paged" else _plain_prompt(s)
    else:
        import speculative_decoding_verify_attn_gb300 as sv

        if op == "logprobs":
            N, K = s["N"], s["K"]
            out = {"logprobs": torch.empty(N, device="cuda"), "entropy": torch.empty(N, device="cuda")}
            if K:
                out["top_ids"] = torch.empty((N, K), dtype=torch.int32, device="cuda")
                out["top_logprobs"] = torch.empty((N, K), device="cuda")
            sv.spec_token_logprobs(s["logits"], s["tokens"], out["logprobs"], entropy=out["entropy"],
                                   top_ids=out.get("top_ids"), top_logprobs=out.get("top_logprobs"))
            return out
        o = torch.empty_like(s["q"])
        if op == "paged":
            sv.spec_paged_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["start"], s["kv_len"], o,
                               max_q=s["max_q"], window=s["window"], k_new=s.get("k_new"), v_new=s.get("v_new"))
        else:
            sv.spec_prefill_attn(s["q"], s["k"], s["v"], s["start"], o, window=s["window"])
    if op == "paged" and s["append"]:
        return {"o": o, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return {"o": o}


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "logprobs":
        N, V, K = case["N"], case["V"], case["K"]
        return {"bytes": N * (V * size + 4 + 8 + 8 * K), "flops": 6.0 * N * V}
    q_len, kv_len = _lengths(case)
    w, D, Hq, Hkv = case["window"], case["D"], case["Hq"], case["Hkv"]
    pairs = keys = 0
    for n, L in zip(q_len, kv_len):
        first = L - n
        if n == 0:
            continue
        keys += L - (max(0, first + 1 - w) if w else 0)
        if w:
            pairs += sum(min(p + 1, w) for p in range(first, L))
        else:
            pairs += n * first + n * (n + 1) // 2
    T = sum(q_len)
    moved = 2 * T * Hq * D + 2 * keys * Hkv * D  # q and o; k and v
    if case.get("append"):
        moved += 2 * T * Hkv * D  # the new rows written (their reads are among the keys)
    return {"bytes": moved * size, "flops": 4.0 * pairs * Hq * D}


def exact(case, seed):
    """The same outputs from the definition in 64 bits, one sequence and key head at a time."""
    if work(case)["flops"] > 4e12 or (case["op"] == "logprobs" and case["N"] * case["V"] > 6e8):
        return None
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        lp, ent, ids, alt = [], [], [], []
        for r in range(0, case["N"], 256):
            x = s["logits"][r: r + 256].double()
            p = torch.softmax(x, 1)
            lse = torch.logsumexp(x, 1, keepdim=True)
            lp.append((x - lse).gather(1, s["tokens"][r: r + 256].long()[:, None])[:, 0])
            ent.append(-torch.xlogy(p, p).sum(1))
            if case["K"]:
                v, i = torch.sort(x, dim=1, descending=True, stable=True)
                ids.append(i[:, : case["K"]].to(torch.int32))
                alt.append(v[:, : case["K"]] - lse)
        out = {"logprobs": torch.cat(lp), "entropy": torch.cat(ent)}
        if case["K"]:
            out["top_ids"], out["top_logprobs"] = torch.cat(ids), torch.cat(alt)
        return out
    q_len, kv_len = _lengths(case)
    Hq, Hkv, D, w = case["Hq"], case["Hkv"], case["D"], case["window"]
    G = Hq // Hkv
    o = torch.zeros((sum(q_len), Hq, D), dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["B"]):
        n, L = q_len[b], kv_len[b]
        if case["op"] == "paged":
            where = torch.arange(L, device="cuda")
            pg, off = s["table"][b].long()[where // case["page"]], where % case["page"]
            if case["append"]:
                s["k_pages"][pg[L - n:], :, off[L - n:]] = s["k_new"][at: at + n]
                s["v_pages"][pg[L - n:], :, off[L - n:]] = s["v_new"][at: at + n]
        step = max(1, (1 << 28) // (L * G))
        for h in range(Hkv):
            if case["op"] == "paged":
                k, v = s["k_pages"][pg, h, off].double(), s["v_pages"][pg, h, off].double()
            else:
                k, v = s["k"][at: at + n, h].double(), s["v"][at: at + n, h].double()
            for r in range(0, n, step):
                e = min(n, r + step)
                q = s["q"][at + r: at + e, h * G: (h + 1) * G].double()
                z = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(D)
                pos = torch.arange(L - n + r, L - n + e, device="cuda")[:, None]
                key = torch.arange(L, device="cuda")[None]
                seen = (key <= pos) & ((key > pos - w) if w else (key >= 0))
                z = z.masked_fill(~seen[:, None], -math.inf)
                o[at + r: at + e, h * G: (h + 1) * G] = torch.softmax(z, -1) @ v
        at += n
    out = {"o": o}
    if case["op"] == "paged" and case["append"]:
        out["k_pages"], out["v_pages"] = s["k_pages"].double(), s["v_pages"].double()
    return out
