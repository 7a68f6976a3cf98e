"""Workloads of the operators around a paged KV cache, for measurement.

Five operators, each with a plain form in elementary torch operations and the library's own call:

* ``rotary``: rotary positions of queries and keys, both layouts, part of the head, scaled for long
  contexts (``spec_rotary``);
* ``append8``: new K/V rows written into a paged cache held in 8 bits with a power-of-two scale for
  each block of tokens and head (``spec_kv8_append``);
* ``paged8``: attention of a ragged batch of new-token chunks over such a cache
  (``spec_paged_attn8``), optionally appending the chunk's K/V in the same call;
* ``fork``: sequences of a paged cache forked, freed and grown, with pages that several sequences hold
  copied before they are written (``spec_page_fork``);
* ``compact``: the pages in use moved to the lowest ids (``spec_page_compact``).

A case is a dict of plain values; lengths and the sharing of pages are drawn from the case alone, values
from the seed.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # the verified rows of one round: 8 sequences of 5 tokens, whole head, halves
        dict(name="rotary-round", op="rotary", dtype="bf16", T=40, Hq=32, Hkv=8, D=128, rot=128, layout="half",
             base=500000.0, factor=1.0, top=32768),
        # a packed prompt batch at far positions: interleaved pairs in part of the head, linearly scaled
        dict(name="rotary-prompt", op="rotary", dtype="bf16", T=16384, Hq=32, Hkv=8, D=128, rot=64, layout="pairs",
             base=10000.0, factor=8.0, top=1000000),
        # the rows of one verify round written into half-filled blocks
        dict(name="append8-round", op="append8", dtype="bf16", B=8, Hkv=8, D=128, q_lo=5, q_hi=5, ctx_lo=1000,
             ctx_hi=4000, page=64, block=16),
        # a ragged batch of prompts written into fresh pages
        dict(name="append8-prompts", op="append8", dtype="bf16", B=16, Hkv=8, D=128, q_lo=60, q_hi=2000, ctx_lo=60,
             ctx_hi=2000, page=64, block=32),
        # one sequence, one new token, a short context: the latency of a single decode step
        dict(name="paged8-decode-short", op="paged8", B=1, Hq=32, Hkv=8, D=128, q_lo=1, q_hi=1, ctx_lo=300, ctx_hi=300,
             page=16, block=16, window=0, append=True),
        # a verify round of 8 sequences (gamma 4, so 5 tokens each) at 16K-32K context, K/V appended
        dict(name="paged8-verify-8b", op="paged8", B=8, Hq=32, Hkv=8, D=128, q_lo=5, q_hi=5, ctx_lo=16384, ctx_hi=32768,
             page=64, block=64, window=0, append=True),
        # continuous batching, head size 64: sequences that decode, verify, rest or take a prompt chunk
        dict(name="paged8-mixed", op="paged8", B=24, Hq=16, Hkv=4, D=64, q_lo=0, q_hi=384, ctx_lo=200, ctx_hi=8192,
             page=32, block=8, window=0, append=True),
        # one 2048-token chunk of a long prompt
        dict(name="paged8-chunk-32k", op="paged8", B=1, Hq=32, Hkv=8, D=128, q_lo=2048, q_hi=2048, ctx_lo=32768,
             ctx_hi=32768, page=64, block=32, window=0, append=False),
        # a serving step of 8 sequences that stay and grow by a round's tokens
        dict(name="fork-round", op="fork", groups=8, width=1, prompt=1000, page=16, spare=400, grow=5, drop=0.0, layers=2,
             Hkv=8, D=128, dtype="e4m3"),
        # 16 prompts of 8 beams: every beam goes on from one of its prompt's, a few are finished
        dict(name="fork-beams", op="fork", groups=16, width=8, prompt=8192, page=64, spare=1000, grow=1, drop=0.05,
             layers=4, Hkv=8, D=128, dtype="bf16"),
        # a small pool after a burst of short sequences
        dict(name="compact-small", op="compact", pages=500, live=0.4, rows=16, page=16, layers=2, Hkv=8, D=128,
             dtype="e4m3"),
        # a large pool that is to give back half of its memory
        dict(name="compact-large", op="compact", pages=8000, live=0.5, rows=256, page=64, layers=4, Hkv=8, D=128,
             dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append8", "paged8", "paged8", "fork", "compact"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 8])
    D = rng.choice([64, 128, 128])
    if op == "rotary":
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), T=_log_uniform(rng, 1, 8192), Hq=Hkv * G, Hkv=Hkv,
                    D=D, rot=rng.choice([D, D, D // 2, D // 4, D - 12]), layout=rng.choice(["half", "pairs"]),
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 32.0]),
                    top=_log_uniform(rng, 1000, 2000000))
    page = rng.choice([16, 24, 32, 64, 128])
    block = rng.choice([1, 2, 4, 8, 8, 12 if page == 24 else 16, page, page])
    if op == "append8":
        q_hi = _log_uniform(rng, 1, 2000)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=_log_uniform(rng, 1, 32), Hkv=Hkv, D=D,
                    q_lo=max(1, q_hi // 4), q_hi=q_hi, ctx_lo=q_hi, ctx_hi=max(q_hi, _log_uniform(rng, 16, 4096)),
                    page=page, block=block)
    if op == "paged8":
        ctx = _log_uniform(rng, 64, 65536)
        q_hi = min(ctx, _log_uniform(rng, 1, 1024))
        B = max(1, min(_log_uniform(rng, 1, 32), (1 << 28) // (ctx * q_hi * Hkv * G // 4 + ctx * Hkv * D)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, q_lo=q_hi if rng.random() < 0.5 else min(1, q_hi), q_hi=q_hi,
                    ctx_lo=max(q_hi, ctx // 3), ctx_hi=ctx, page=page, block=block,
                    window=rng.choice([0, 0, 0, 128, 512]), append=rng.random() < 0.5)
    dtype = rng.choice(["e4m3", "bf16"])
    layers = rng.choice([1, 2, 4])
    if op == "fork":
        groups, width, grow = _log_uniform(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.choice([0, 1, 5, 40])
        return dict(op=op, groups=groups, width=width, prompt=_log_uniform(rng, 20, 8192), page=page,
                    spare=groups * width * (3 + grow // page) + _log_uniform(rng, 1, 500), grow=grow,
                    drop=rng.choice([0.0, 0.1, 0.5]), layers=layers, Hkv=Hkv, D=D, dtype=dtype)
    return dict(op=op, pages=_log_uniform(rng, 10, 8000 * 64 // max(64, page)), live=rng.choice([0.05, 0.3, 0.7, 0.95]),
                rows=_log_uniform(rng, 1, 256), page=page, layers=layers, Hkv=Hkv, D=D, dtype=dtype)


def _lengths(case):
    """New tokens and context length (new ones included) of each sequence, from the case alone."""
    rng = random.Random("%s/%s/%s/%s" % (case["B"], case["q_lo"], case["q_hi"], case["ctx_hi"]))
    B, lo, hi = case["B"], case["q_lo"], case["q_hi"]
    if lo == 0:  # rest, decode, verify, or a chunk of the prompt
        q = [rng.choice([0, 1, 1, 5, 5, rng.randint(16, hi), hi]) for _ in range(B)]
        q[0], q[-1] = hi, 1
    else:
        q = [rng.randint(lo, hi) for _ in range(B)]
    if case["op"] == "append8" and lo > 5:  # prompts into fresh pages
        return q, list(q)
    return q, [max(n, rng.randint(case["ctx_lo"], case["ctx_hi"])) for n in q]


def _beams(case):
    """Rows of a beam search before a step, from the case alone: page ids, lengths, parents, growth and
    the number of holders of each page."""
    rng = random.Random("fork/%s/%s/%s/%s" % (case["groups"], case["width"], case["prompt"], case["page"]))
    size, W = case["page"], case["width"]
    rows, lens, parent, grow, top = [], [], [], [], 0
    for g in range(case["groups"]):
        prompt = rng.randint(max(1, case["prompt"] // 2), case["prompt"])
        shared = list(range(top, top + prompt // size))
        top += len(shared)
        more = rng.randint(1, 100)
        tail = -(-(prompt + more) // size) - len(shared)
        for w in range(W):
            if w and rng.random() < 0.3:  # forked in the step before: the last pages are shared too
                rows.append(list(rows[-1]))
            else:
                rows.append(shared + list(range(top, top + tail)))
                top += tail
            lens.append(prompt + more)
            gone = rng.random() < case["drop"]
            parent.append(-1 if gone else g * W + rng.randrange(W))
            grow.append(0 if gone else case["grow"])
    pages = top + case["spare"]
    order = list(range(pages))
    rng.shuffle(order)
    rows = [[order[p] for p in r] for r in rows]
    refs = [0] * pages
    for r in rows:
        for p in r:
            refs[p] += 1
    for r in rows[::3]:  # a prefix cache of the caller holds some prompts' first pages as well
        refs[r[0]] += 1
    cols = max(len(r) for r in rows) + -(-case["grow"] // size) + 3
    return rows, lens, parent, grow, refs, cols


def _pool(case):
    """Pages of the rows of a pool with gaps, from the case alone, and the holders of each page."""
    rng = random.Random("compact/%s/%s/%s" % (case["pages"], case["rows"], case["live"]))
    used = rng.sample(range(case["pages"]), max(1, int(case["pages"] * case["live"])))
    cuts = sorted(rng.randrange(len(used) + 1) for _ in range(case["rows"] - 1))
    rows = [used[a:b] for a, b in zip([0] + cuts, cuts + [len(used)])]
    for r in rows[1::2]:  # a common prefix
        r[:0] = rows[0][:2]
    refs = [0] * case["pages"]
    for r in rows:
        for p in r:
            refs[p] += 1
    return rows, refs


def _tables(rows, cols):
    table = torch.zeros((len(rows), cols), dtype=torch.int32)
    for b, r in enumerate(rows):
        table[b, : len(r)] = torch.tensor(r, dtype=torch.int32)
    return table.cuda(), _ints([len(r) for r in rows])


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="bf16", scale=1.0):
        kept = torch.float32 if dtype == "f32" else torch.bfloat16
        return torch.empty(shape, dtype=kept, device="cuda").normal_(0.0, scale, generator=g).to(DTYPES[dtype])

    s = dict(case)
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    if op == "rotary":
        T, rot = case["T"], case["rot"]
        s["q"], s["k"] = (normal(T, H, D, dtype=case["dtype"]) for H in (case["Hq"], Hkv))
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        first = torch.randint(0, case["top"], (-(-T // 64),), generator=g, device="cuda")
        s["positions"] = (first[:, None] + torch.arange(64, device="cuda")).reshape(-1)[:T].to(torch.int32)
        # the part of a turn that a position adds, in units of 2^-64 turns
        turn = [case["base"] ** (-2.0 * i / rot) / case["factor"] / (2.0 * math.pi) for i in range(rot // 2)]
        s["steps"] = torch.tensor([int(x * 2.0 ** 64) for x in turn], dtype=torch.int64, device="cuda")
        return s
    if op in ("fork", "compact"):
        if op == "fork":
            rows, lens, parent, grow, refs, cols = _beams(case)
            s["kv_len"], s["parent"], s["grow_by"] = _ints(lens), _ints(parent), _ints(grow)
            s["len_out"] = torch.zeros_like(s["kv_len"])
        else:
            rows, refs = _pool(case)
            cols = max(len(r) for r in rows) + 3
            s["moved"], s["live_out"] = _ints([0] * len(refs)), _ints([0])
        s["table"], s["held"] = _tables(rows, cols)
        s["refs"] = _ints(refs)
        s["table_out"], s["held_out"] = torch.zeros_like(s["table"]), torch.zeros_like(s["held"])
        s["refs_out"] = torch.zeros_like(s["refs"])
        shape = (len(refs), Hkv, case["page"], D)
        s["caches"] = [normal(*shape, dtype=case["dtype"]) for _ in range(2 * case["layers"])]
        if case["dtype"] == "e4m3":
            s["caches"] += [torch.randint(100, 140, (len(refs), Hkv, 2), generator=g, device="cuda", dtype=torch.uint8)
                            for _ in range(2 * case["layers"])]
        return s
    q_len, kv_len = _lengths(case)
    B, T, page, block = case["B"], sum(q_len), case["page"], case["block"]
    s["max_q"] = max(q_len)
    s["start"] = _ints([sum(q_len[:b]) for b in range(B + 1)])
    per = [-(-n // page) for n in kv_len]
    pages = sum(per) + 3
    # what the cache holds: values that fill e4m3's range, with scales that differ from block to block
    s["k_pages"], s["v_pages"] = (normal(pages, Hkv, page, D, dtype="e4m3", scale=60.0) for _ in range(2))
    s["k_exp"], s["v_exp"] = (
        (120 + torch.randint(0, 3, (pages, Hkv, page // block), generator=g, device="cuda")).to(torch.uint8)
        for _ in range(2))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.zeros((B, max(per)), dtype=torch.int32, device="cuda")
    for b in range(B):
        s["table"][b, : per[b]] = order[sum(per[:b]): sum(per[: b + 1])]
    s["kv_len"] = _ints(kv_len)
    if op == "append8" or case["append"]:
        # a few channels of keys are far larger than the others
        s["k_new"], s["v_new"] = (normal(T, Hkv, D, dtype=case.get("dtype", "bf16")) for _ in range(2))
        s["k_new"][:, :, ::37] *= 8
    if op == "paged8":
        s["q"] = normal(T, case["Hq"], D)
    return s


# ------------------------------------------------------------------------------ plain forms
def _of_token(start, T):
    """Sequence and index in it of each packed token."""
    t = torch.arange(T, device=start.device)
    seq = torch.searchsorted(start[1:].long(), t, right=True)
    return seq, t - start.long()[seq]


def _plain_rotary(s):
    rot, D = s["rot"], s["D"]
    # in 64 bits: far positions take many turns
    turn = s["positions"].double()[:, None] * (s["steps"].double() * 2.0 ** -64)
    angle = (turn - turn.floor()) * (2.0 * math.pi)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        y = x.float()
        r = y[..., :rot]
        if s["layout"] == "half":
            a, b = r[..., : rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return (torch.cat((r, y[..., rot:]), -1) if rot < D else r).to(x.dtype)

    return {"q": turned(s["q"]), "k": turned(s["k"])}


def _needed_exponent(x):
    """The least exponent, plus 127, whose scale brings x, the largest magnitude of a block, within 448."""
    m, e = torch.frexp(x)
    return torch.where(x > 0, (e - torch.where(m <= 0.875, 9, 8)).clamp(-64, 64), -64) + 127


def _plain_append8(s):
    start, table, page, block = s["start"].long(), s["table"].long(), s["page"], s["block"]
    T = s["k_new"].shape[0]
    seq, j = _of_token(start, T)
    n = start[1:] - start[:-1]
    kv_len = s["kv_len"].long()
    first = kv_len - n
    pos = first[seq] + j
    at, slot = table[seq, pos // page], pos % page
    # the tokens of a block that were there before: those of the block of the sequence's first new token
    old = (first // block * block)[:, None] + torch.arange(block, device=start.device)
    seen = (old < first[:, None]) & (n > 0)[:, None]
    old = torch.where(seen, old, 0)
    begin = torch.where(n > 0, first, 0)
    old_at, old_slot = table.gather(1, old // page), old % page
    edge_at, edge_blk = table.gather(1, (begin // page)[:, None])[:, 0], begin % page // block
    live = seen.any(1)
    for x, pages, exp in ((s["k_new"], s["k_pages"], s["k_exp"]), (s["v_new"], s["v_pages"], s["v_exp"])):
        y = x.float()
        P, Hkv, per = exp.shape
        where = at * per + slot // block  # the block of each new token
        need = _needed_exponent(y.abs().amax(2))
        before = exp[edge_at, :, edge_blk].int()  # [B, Hkv]
        flat = torch.zeros((P * per, Hkv), dtype=torch.int32, device=x.device)
        flat.scatter_reduce_(0, where[:, None].expand(-1, Hkv), need.int(), "amax")
        edge = edge_at * per + edge_blk
        flat.scatter_reduce_(0, edge[:, None].expand(-1, Hkv), torch.where(live[:, None], before, 0), "amax")
        after = flat[edge]
        grown = flat.view(P, per, Hkv).transpose(1, 2)
        exp.copy_(torch.where(grown > 0, grown, exp.int()).to(torch.uint8))
        # old tokens at the block's new scale
        was = pages.view(torch.uint8)[old_at, :, old_slot].view(pages.dtype).float()  # [B, block, Hkv, D]
        moved = torch.ldexp(was, (before - after)[:, None, :, None])
        keep = torch.where(seen[:, :, None, None], moved.to(pages.dtype).float(), was)
        rows = seen.nonzero(as_tuple=True)
        pages.view(torch.uint8)[old_at[rows], :, old_slot[rows]] = keep[rows].to(pages.dtype).view(torch.uint8)
        scaled = torch.ldexp(y, (127 - flat[where])[:, :, None]).clamp(-448.0, 448.0)
        pages.view(torch.uint8)[at, :, slot] = scaled.to(pages.dtype).view(torch.uint8)


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


def _plain_paged8(s):
    if s["append"]:
        _plain_append8(s)
    start, table, block = s["start"].long(), s["table"].long(), s["block"]
    seq, j = _of_token(start, s["q"].shape[0])
    n = start[1:] - start[:-1]
    kv_len = s["kv_len"].long()

    def cache(pages, exp):
        got = pages.view(torch.uint8)[table].view(pages.dtype).float()  # [B, pages, Hkv, page, D]
        e = exp[table].int().repeat_interleave(block, 3) - 127
        got = torch.ldexp(got, e[..., None])
        return got.permute(0, 2, 1, 3, 4).reshape(table.shape[0], pages.shape[1], -1, pages.shape[3])

    m = s["max_q"]
    rows = torch.arange(m, device=start.device)
    q_pos = torch.where(rows < n[:, None], (kv_len - n)[:, None] + rows, -1)
    q = s["q"][(start[:-1, None] + rows).clamp(max=s["q"].shape[0] - 1)].float()
    o = _attend(q, cache(s["k_pages"], s["k_exp"]), cache(s["v_pages"], s["v_exp"]), q_pos, kv_len, s["window"])
    return o[seq, j].to(s["q"].dtype)


def _raw(cache):
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _plain_fork(s):
    table, size, refs = s["table"].long(), s["page"], s["refs"]
    B, cols = table.shape
    P = refs.shape[0]
    goes = s["parent"] >= 0
    parent = s["parent"].long().clamp(min=0)
    before = torch.where(goes, s["kv_len"].long()[parent], 0)
    grow = torch.where(goes, s["grow_by"].long(), 0)
    kept, need = (before + size - 1) // size, (before + grow + size - 1) // size
    col, row = torch.arange(cols, device=table.device), torch.arange(B, device=table.device)
    held, keep = col < s["held"][:, None], col < kept[:, None]
    source = table[parent]
    count = refs.long().index_add(0, torch.where(held, table, 0).flatten(), -held.long().flatten())
    count.index_add_(0, torch.where(keep, source, 0).flatten(), keep.long().flatten())
    # a last page that is written to and held by others: copied, but for the lowest row if all holders write
    writes = goes & (grow > 0) & (before % size != 0)
    last = torch.where(writes, source.gather(1, (before // size).clamp(max=cols - 1)[:, None])[:, 0], 0)
    writers = torch.zeros(P, dtype=torch.long, device=table.device).index_add(0, last, writes.long())
    lowest = torch.full((P,), B, device=table.device).scatter_reduce(0, last, torch.where(writes, row, B), "amin")
    copies = writes & (count[last] > 1) & ~((writers[last] == count[last]) & (lowest[last] == row))
    fresh = copies.long() + need - kept
    at = (fresh.cumsum(0) - fresh)[:, None]
    free = torch.sort((count > 0).int(), stable=True).indices  # free pages, in ascending order, come first
    new = free[(at + copies.long()[:, None] + col - kept[:, None]).clamp(0, P - 1)]
    own_copy = copies[:, None] & (col == (before // size)[:, None])
    new = torch.where(own_copy, free[at.clamp(max=P - 1)], torch.where(keep, source, new))
    used = col < need[:, None]
    s["table_out"].copy_(torch.where(used, new, s["table_out"].long()))
    s["held_out"].copy_(need)
    s["len_out"].copy_(before + grow)
    count.index_add_(0, last, -copies.long())
    count.index_add_(0, torch.where(used, new, 0).flatten(), (used & (own_copy | ~keep)).long().flatten())
    s["refs_out"].copy_(count)
    which = copies.nonzero()[:, 0]
    to = free[at[which, 0]]
    for c in s["caches"]:
        _raw(c)[to] = _raw(c)[last[which]]


def _plain_compact(s):
    refs = s["refs"]
    page = torch.arange(refs.shape[0], device=refs.device)
    used = refs > 0
    live = used.sum()
    gaps, tails = (~used & (page < live)).nonzero()[:, 0], (used & (page >= live)).nonzero()[:, 0]
    moved = torch.where(used, page, -1)
    moved[tails] = gaps
    table = s["table"].long()
    inside = torch.arange(table.shape[1], device=refs.device) < s["held"][:, None]
    s["table_out"].copy_(torch.where(inside, moved[table], s["table_out"].long()))
    count = torch.where(page < live, refs, 0)
    count[gaps] = refs[tails]
    s["refs_out"].copy_(count)
    s["moved"].copy_(moved)
    s["live_out"].copy_(live)
    for c in s["caches"]:
        _raw(c)[gaps] = _raw(c)[tails]


def run(s):
    op = s["op"]
    if not own:
        if op == "rotary":
            return _plain_rotary(s)
        if op == "append8":
            _plain_append8(s)
        elif op == "paged8":
            o = _plain_paged8(s)
        elif op == "fork":
            _plain_fork(s)
        else:
            _plain_compact(s)
    else:
        import speculative_decoding_verify_attn_gb300 as sv

        if op == "rotary":
            sv.spec_rotary(s["q"], s["k"], s["steps"], positions=s["positions"], q_out=s["q_out"], k_out=s["k_out"],
                           layout=sv.SPEC_ROTARY_HALF if s["layout"] == "half" else sv.SPEC_ROTARY_PAIRS)
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append8":
            sv.spec_kv8_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"], s["table"],
                               s["start"], s["kv_len"])
        elif op == "paged8":
            o = torch.empty_like(s["q"])
            sv.spec_paged_attn8(s["q"], s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"], s["table"], s["start"],
                                s["kv_len"], o, max_q=s["max_q"], window=s["window"], k_new=s.get("k_new"),
                                v_new=s.get("v_new"))
        elif op == "fork":
            sv.spec_page_fork(s["table"], s["held"], s["kv_len"], s["refs"], s["parent"], page_size=s["page"],
                              grow=s["grow_by"], caches=s["caches"], table_out=s["table_out"], held_out=s["held_out"],
                              len_out=s["len_out"], refs_out=s["refs_out"])
        else:
            sv.spec_page_compact(s["table"], s["held"], s["refs"], caches=s["caches"], table_out=s["table_out"],
                                 refs_out=s["refs_out"], moved=s["moved"], num_live=s["live_out"])
    if op == "fork":
        return {"table": s["table_out"], "held": s["held_out"], "kv_len": s["len_out"], "refs": s["refs_out"],
                "caches": s["caches"]}
    if op == "compact":
        return {"table": s["table_out"], "refs": s["refs_out"], "moved": s["moved"], "live": s["live_out"],
                "caches": s["caches"]}
    out = {"o": o} if op == "paged8" else {}
    if op == "append8" or s["append"]:
        out.update({x: s[x] for x in ("k_pages", "v_pages", "k_exp", "v_exp")})
    return out


def _page_bytes(case):
    """Bytes of one page in all arrays of the cache."""
    values = 2 * case["layers"] * case["Hkv"] * case["page"] * case["D"]
    return values * 2 if case["dtype"] == "bf16" else values + 2 * case["layers"] * case["Hkv"] * 2


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    if op == "rotary":
        size = 2 if case["dtype"] == "bf16" else 4
        heads = case["Hq"] + Hkv
        return {"bytes": case["T"] * (2 * heads * D * size + 4) + 4 * case["rot"],
                "flops": 3.0 * case["T"] * heads * case["rot"]}
    if op == "fork":
        rows, lens, parent, grow, refs, _ = _beams(case)
        size, held = case["page"], [0] * len(refs)
        for b, r in zip(parent, grow):
            for p in rows[b] if b >= 0 else ():
                held[p] += 1
        copies = writers = 0
        seen = {}
        for b, n in zip(parent, grow):
            if b >= 0 and n and lens[b] % size:
                last = rows[b][lens[b] // size]
                seen[last] = seen.get(last, 0) + 1
        for last, n in seen.items():
            copies += n if held[last] > n else n - 1
        entries = sum(len(rows[b]) for b in parent if b >= 0)
        return {"bytes": 8 * entries + 8 * len(refs) + 24 * len(rows) + 2 * copies * _page_bytes(case), "flops": 0.0}
    if op == "compact":
        rows, refs = _pool(case)
        live = sum(n > 0 for n in refs)
        moves = sum(n > 0 for n in refs[live:])
        return {"bytes": 8 * sum(map(len, rows)) + 12 * len(refs) + 2 * moves * _page_bytes(case), "flops": 0.0}
    q_len, kv_len = _lengths(case)
    T, block = sum(q_len), case["block"]
    size = 4 if case.get("dtype") == "f32" else 2
    written = 2 * T * Hkv * D + 2 * Hkv * sum(-(-n // block) for n in q_len)
    if op == "append8":
        return {"bytes": 2 * T * Hkv * D * size + written, "flops": 4.0 * T * Hkv * D}
    w, Hq = case["window"], case["Hq"]
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
    moved = 4 * T * Hq * D + 2 * Hkv * (keys * D + keys // block)  # q and o; k, v and their scales
    if case["append"]:
        moved += written + 2 * T * Hkv * D  # the new rows are read in 16 bits instead of 8
    return {"bytes": moved, "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------------------ the definition in 64 bits
def _exact_append(case, s, q_len, kv_len):
    """The cache after the append, one sequence, block and head at a time."""
    page, block = case["page"], case["block"]
    table = s["table"].tolist()
    row = 0
    for b in range(case["B"]):
        for x, pages, exp in (("k_new", "k_pages", "k_exp"), ("v_new", "v_pages", "v_exp")):
            first, end = kv_len[b] - q_len[b], kv_len[b]
            for t0 in range(first // block * block, end, block):
                lo, hi = max(t0, first), min(t0 + block, end)
                if hi <= lo:
                    continue
                pg, off = table[b][t0 // page], t0 % page
                new = s[x][row + lo - first: row + hi - first].double()  # [tokens, Hkv, D]
                top = new.abs().amax((0, 2))
                e = torch.ceil(torch.log2(top / 448.0)).clamp(-64, 64)
                e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e)
                e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e).clamp(-64, 64)
                e = torch.where(top > 0, e, -64.0)
                if lo > t0:
                    was = exp_of(s[exp], pg, off // block)
                    e = torch.maximum(e, was)
                    old = s[pages][pg, :, off: off + lo - t0].double() * torch.exp2(was - e)[:, None, None]
                    s[pages][pg, :, off: off + lo - t0] = old.float().to(torch.float8_e4m3fn)
                s[exp][pg, :, off // block] = (e + 127).to(torch.uint8)
                q = (new.transpose(0, 1) * torch.exp2(-e)[:, None, None]).clamp(-448, 448)
                s[pages][pg, :, off + lo - t0: off + hi - t0] = q.float().to(torch.float8_e4m3fn)
        row += q_len[b]


def exp_of(exp, page, block):
    return exp[page, :, block].double() - 127.0


def exact(case, seed):
    """The same outputs from the definition in 64 bits; none for page ids, counts and moved pages."""
    op = case["op"]
    if op in ("fork", "compact") or work(case)["flops"] > 4e12:
        return None
    Hkv, D = case["Hkv"], case["D"]
    if op == "rotary":
        s = prepare(case, seed)
        rot, out = case["rot"], {}
        i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
        angle = s["positions"].double()[:, None] * (case["base"] ** (-2.0 * i / rot) / case["factor"])
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for x in ("q", "k"):
            y = s[x].double()
            if case["layout"] == "half":
                z = torch.complex(y[..., : rot // 2], y[..., rot // 2: rot]) * turn
                y = torch.cat((z.real, z.imag, y[..., rot:]), -1)
            else:
                z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
                y = torch.cat((torch.view_as_real(z).flatten(-2), y[..., rot:]), -1)
            out[x] = y
        return out
    q_len, kv_len = _lengths(case)
    appends = op == "append8" or case["append"]
    if appends and sum(q_len) // case["block"] + case["B"] > 4000:
        return None
    s = prepare(case, seed)
    if appends:
        _exact_append(case, s, q_len, kv_len)
    out = {}
    if appends:
        out = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double(), "k_exp": None, "v_exp": None}
    if op == "append8":
        return out
    Hq, w = case["Hq"], case["window"]
    G, page, block = Hq // Hkv, case["page"], case["block"]
    o = torch.zeros((sum(q_len), Hq, D), dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["B"]):
        n, L = q_len[b], kv_len[b]
        where = torch.arange(L, device="cuda")
        pg, off = s["table"][b].long()[where // page], where % page
        step = max(1, (1 << 28) // (L * G))
        for h in range(Hkv if n else 0):
            k, v = (s[x + "_pages"].view(torch.uint8)[pg, h, off].view(torch.float8_e4m3fn).double()
                    * torch.exp2(s[x + "_exp"][pg, h, off // block].double() - 127.0)[:, None] for x in "kv")
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
    return {"o": o, **out}
