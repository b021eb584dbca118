"""The operators of a paged KV cache and of draft verification, as they are measured.

A step of a serving loop over a paged cache is: ``plan`` (block tables and slot
maps on the GPU from the request lengths), then per layer ``qk_norm_rope``
(norms of queries and keys for each head and the position rotation in one
pass, keys and values stored in their pages) and ``attention`` (of the new
tokens over the pages), and at the end, where the new tokens were drafted,
``verify`` (the drafts against the target's probabilities, from given random
numbers).

``run`` computes an operator in its plain form with elementary torch
operations, or, where ``own`` is true, calls the framework's operators.
"""
from __future__ import annotations

import random

import torch

own = False

DEV = "cuda"
EPS = 1e-5
THETA = 5e5


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # eight requests in decode, one new token each: what every step pays before its first layer
        dict(name="plan_decode", op="plan", B=8, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=1, page=16, back=1, pad=0,
             lens=1),
        # a full server: prompts being filled in beside decodes, some requests finished or rolled back, a padded batch
        dict(name="plan_mixed", op="plan", B=509, ctx_lo=0, ctx_hi=8192, new_lo=0, new_hi=256, page=16, back=64, pad=100,
             lens=2),
        # one token of one request, from the decoder's f32 activations
        dict(name="norm_rope_token", op="norm_rope", N=1, pad=0, Hq=32, Hkv=8, D=128, page=64, dtype="f32", norm=True,
             far=8192, lens=1),
        # a ragged chunk far into a long context, a padded batch, seven query heads per key head, f32
        dict(name="norm_rope_chunk", op="norm_rope", N=777, pad=23, Hq=28, Hkv=4, D=128, page=16, dtype="f32", norm=True,
             far=1000000, lens=2),
        # a whole prompt from 16-bit activations
        dict(name="norm_rope_prompt", op="norm_rope", N=8192, pad=0, Hq=32, Hkv=8, D=128, page=64, dtype="bf16",
             norm=True, far=32768, lens=3),
        # the single token of the 8B-shaped decode workload, KV 4096
        dict(name="attention_token", op="attention", B=1, ctx_lo=4096, ctx_hi=4096, new_lo=1, new_hi=1, Hq=32, Hkv=8,
             D=128, page=64, pad=0, lens=1),
        # a decode batch over the ragged workload's lengths, small pages
        dict(name="attention_decode", op="attention", B=64, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=1, Hq=32, Hkv=8,
             D=128, page=16, pad=0, lens=2),
        # five drafted tokens of each of the four long-context sequences
        dict(name="attention_drafts", op="attention", B=4, ctx_lo=32768, ctx_hi=32768, new_lo=5, new_hi=5, Hq=32, Hkv=8,
             D=128, page=128, pad=0, lens=3),
        # chunks of several requests, odd lengths, 64-wide heads, a padded batch
        dict(name="attention_chunks", op="attention", B=7, ctx_lo=0, ctx_hi=3001, new_lo=1, new_hi=701, Hq=32, Hkv=4,
             D=64, page=32, pad=17, lens=4),
        # a whole prompt
        dict(name="attention_prompt", op="attention", B=1, ctx_lo=0, ctx_hi=0, new_lo=8192, new_hi=8192, Hq=32, Hkv=8,
             D=128, page=64, pad=0, lens=5),
        # one sequence's four drafts
        dict(name="verify_one", op="verify", B=1, K=4, V=128256, q=True, ragged=False, lens=1),
        # a batch of speculating requests with drafts of different lengths
        dict(name="verify_batch", op="verify", B=64, K=7, V=128256, q=True, ragged=True, lens=2),
    ]


HEADS = [(32, 8, 128), (28, 4, 128), (40, 8, 128), (8, 1, 128), (64, 8, 128), (4, 2, 64), (32, 4, 64), (12, 12, 64)]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random() + rng.random())))


def _draw(rng):
    op = rng.choice(["plan", "norm_rope", "attention", "attention", "attention", "verify"])
    lens = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    pad = rng.choice([0, 0, rng.randrange(1, 65)])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 512), ctx_lo=0, ctx_hi=_log(rng, 64, 8192), new_lo=0, new_hi=_log(rng, 1, 256),
                    page=page, back=rng.choice([1, 16, 64]), pad=pad, lens=lens)
    Hq, Hkv, D = rng.choice(HEADS)
    if op == "norm_rope":
        return dict(op=op, N=_log(rng, 1, 8192), pad=pad, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    dtype=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.75, far=_log(rng, 16384, 1000000), lens=lens)
    if op == "verify":
        return dict(op=op, B=_log(rng, 1, 64), K=rng.randrange(1, 9), V=_log(rng, 1000, 128256),
                    q=rng.random() < 0.75, ragged=rng.random() < 0.5, lens=lens)
    kind = rng.choice(["decode", "drafts", "chunks", "prompt"])
    if kind == "decode":
        shape = dict(B=_log(rng, 1, 96), new_lo=1, new_hi=1, ctx_lo=rng.choice([0, 512]), ctx_hi=_log(rng, 600, 32768))
    elif kind == "drafts":
        shape = dict(B=_log(rng, 1, 32), new_lo=rng.choice([0, 1]), new_hi=rng.randrange(2, 9),
                     ctx_lo=rng.choice([0, 512]), ctx_hi=_log(rng, 600, 32768))
    elif kind == "chunks":
        shape = dict(B=rng.randrange(2, 12), new_lo=rng.choice([0, 1, 64]), new_hi=_log(rng, 65, 1024), ctx_lo=0,
                     ctx_hi=_log(rng, 64, 4096))
    else:
        n = _log(rng, 256, 8192)
        shape = dict(B=1, new_lo=n, new_hi=n, ctx_lo=0, ctx_hi=rng.choice([0, 0, 1000]))
    return dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=page, pad=pad, lens=lens, **shape)


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("plan", "norm_rope", "attention", "verify")}
    while True:
        c = _draw(rng)
        if _cost(c) > most[c["op"]]:
            continue
        if c["op"] == "attention":  # the plain form holds every score of a padded batch
            ctx, new = _lengths(c)
            far = max(a + b for a, b in zip(ctx, new))
            if max(new) < 1 or c["B"] * c["Hq"] * max(new) * far > 1 << 31 or c["B"] * c["Hkv"] * c["D"] * far > 1 << 30:
                continue
        return c


def _lengths(c):
    """(cached tokens, new tokens) of every request: the case's own, whatever the seed."""
    r = random.Random(c["lens"])
    return ([r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["B"])],
            [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])])


def _pages(n, page):
    return -(-n // page)


def _held(c):
    """Pages each request holds before the step: what its cached tokens need, or more where drafts were rolled back
    or the request has finished (no cached and no new tokens; its pages go back)."""
    r = random.Random(c["lens"] + 1)
    ctx, new = _lengths(c)
    held = []
    for b in range(c["B"]):
        more = r.randint(0, 3) if r.random() < 0.2 and c["back"] > 1 else 0
        held.append(_pages(ctx[b], c["page"]) + more)
    if c["back"] > 1:
        for b in range(c["back"] - 1, c["B"], c["back"]):
            ctx[b], new[b] = 0, 0
    return ctx, new, held


def work(case):
    c = case
    if c["op"] == "plan":
        ctx, new, held = _held(c)
        want = [_pages(a + b, c["page"]) for a, b in zip(ctx, new)]
        n = sum(new)
        grown = sum(max(0, w - h) for w, h in zip(want, held))
        back = sum(max(0, h - w) for w, h in zip(want, held))
        touched = sum(_pages(a + b, c["page"]) - a // c["page"] for a, b in zip(ctx, new) if b)
        # lengths and held pages in, cu and held pages out; positions and slots; pages looked up and moved
        return {"bytes": 4 * (5 * c["B"] + 2 * (n + c["pad"]) + touched + 2 * grown + 2 * back), "flops": 0}
    if c["op"] == "norm_rope":
        n = c["N"]
        size = 4 if c["dtype"] == "f32" else 2
        width = (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": n * width * (size + 2) + 8 * (n + c["pad"]) + 4 * c["D"],
                "flops": n * (c["Hq"] + c["Hkv"]) * c["D"] * (7 if c["norm"] else 3)}
    if c["op"] == "attention":
        ctx, new = _lengths(c)
        keys = sum(a + b for a, b in zip(ctx, new) if b)
        pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, new))
        n = sum(new)
        return {"bytes": keys * c["Hkv"] * c["D"] * 4 + n * c["Hq"] * c["D"] * 4
                + 4 * sum(_pages(a + b, c["page"]) for a, b in zip(ctx, new)) + 8 * c["B"],
                "flops": 4 * c["D"] * c["Hq"] * pairs}
    # a request's drafts need K probabilities; its last token one row of the target's and, after a rejection, of the draft's
    rows = 2 if c["q"] else 1
    return {"bytes": c["B"] * (rows * c["V"] * 4 + c["K"] * 20), "flops": 2 * rows * c["B"] * c["V"]}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    return {"plan": _prepare_plan, "norm_rope": _prepare_norm_rope, "attention": _prepare_attention,
            "verify": _prepare_verify}[case["op"]](case, seed)


def _prepare_plan(c, seed):
    ctx, new, held = _held(c)
    want = [_pages(a + b, c["page"]) for a, b in zip(ctx, new)]
    max_pages = max(max(held), max(want)) + 2
    num_pages = sum(held) + sum(max(0, w - h) for w, h in zip(want, held)) + 11
    ids = torch.randperm(num_pages, generator=_gen(seed), device=DEV).to(torch.int32)
    table = torch.full((c["B"], max_pages), -1, dtype=torch.int32, device=DEV)
    own_pages = torch.arange(max_pages, device=DEV)[None, :] < _i32(held)[:, None]
    table[own_pages] = ids[: sum(held)]
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    free[: num_pages - sum(held)] = ids[sum(held):]
    n = sum(new) + c["pad"]
    return dict(c=c, ctx=_i32(ctx), new=_i32(new), held=_i32(held), table=table, free=free,
                count=_i32([num_pages - sum(held)]), held_out=_i32(held), count_out=_i32([0]),
                cu=_i32([0] * (c["B"] + 1)), positions=_i32([0] * n), slots=_i32([0] * n))


def _prepare_norm_rope(c, seed):
    g = _gen(seed)
    n, rows = c["N"], c["N"] + c["pad"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    qkv = torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
    gain = [(1 + 0.02 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
            for _ in range(2)]
    num_pages = _pages(n, c["page"]) + 3
    slots = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    positions = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    # a chunk of consecutive tokens, its pages anywhere in the pool
    first = random.Random(c["lens"]).randrange(0, c["far"] - n + 1)
    first -= first % c["page"]
    ids = torch.randperm(num_pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    slots[:n] = (ids[i // c["page"]] * c["page"] + i % c["page"]).to(torch.int32)
    positions[:n] = (first + i).to(torch.int32)
    pool = [torch.zeros(num_pages, Hkv, c["page"], D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    return dict(c=c, qkv=qkv, q_gamma=gain[0], k_gamma=gain[1], positions=positions, slots=slots, kpool=pool[0],
                vpool=pool[1], q=torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=DEV), n=n)


def _prepare_attention(c, seed):
    g = _gen(seed)
    ctx, new = _lengths(c)
    n, D, page = sum(new), c["D"], c["page"]
    pages = [_pages(a + b, page) for a, b in zip(ctx, new)]
    num_pages, max_pages = sum(pages) + 5, max(pages) + 1
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["B"], max_pages), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max_pages, device=DEV)[None, :] < _i32(pages)[:, None]] = ids[: sum(pages)]
    pool = [torch.randn(num_pages, c["Hkv"], page, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    q = torch.randn(n + c["pad"], c["Hq"], D, generator=g, device=DEV) * 1.5
    cu = [0]
    for b in new:
        cu.append(cu[-1] + b)
    return dict(c=c, q=q.to(torch.bfloat16), kpool=pool[0], vpool=pool[1], table=table, cu=_i32(cu), ctx=_i32(ctx),
                max_new=max(new), far=max(a + b for a, b in zip(ctx, new)),
                out=torch.zeros(n + c["pad"], c["Hq"], D, dtype=torch.bfloat16, device=DEV))


def _prepare_verify(c, seed):
    g = _gen(seed)
    B, K, V = c["B"], c["K"], c["V"]
    r = random.Random(c["lens"])
    logits = torch.randn(B, K + 1, V, generator=g, device=DEV) * 2.5
    p = torch.softmax(logits, -1)
    # the draft model's distribution is near the target's
    near = logits[:, :K] + 0.7 * torch.randn(B, K, V, generator=g, device=DEV)
    q = torch.softmax(near, -1)
    drafts = torch.multinomial(q.view(B * K, V), 1, generator=g).view(B, K).to(torch.int32)
    u = torch.rand(B, K + 1, generator=g, device=DEV)
    length = _i32([r.randint(0, K) if c["ragged"] else K for _ in range(B)])
    return dict(c=c, p=p, q=q if c["q"] else None, drafts=drafts, u=u, length=length)


# ----------------------------------------------------------------- one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return _own(op, state)
    return {"plan": _plain_plan, "norm_rope": _plain_norm_rope, "attention": _plain_attention,
            "verify": _plain_verify}[op](state)


def _own(op, s):
    c = s["c"]
    if op == "verify":
        from task_graph_interpreter_gb300 import speculative
        tokens, accepted = speculative.verify_drafts(s["p"], s["drafts"], s["u"], q=s["q"], draft_len=s["length"])
        return {"tokens": tokens, "accepted": accepted}
    from task_graph_interpreter_gb300 import paged
    if op == "plan":
        paged.plan(s["ctx"], s["new"], s["table"], s["held"], s["free"], s["count"], c["page"], cu=s["cu"],
                   positions=s["positions"], slots=s["slots"], held_out=s["held_out"], count_out=s["count_out"])
        return {k: s[k] for k in ("table", "free", "held_out", "count_out", "cu", "positions", "slots")}
    if op == "norm_rope":
        paged.qk_norm_rope(s["qkv"], c["Hq"], c["Hkv"], c["D"], s["positions"], s["slots"], s["kpool"], s["vpool"],
                           q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS, rope_theta=THETA, out=s["q"])
        return {k: s[k] for k in ("q", "kpool", "vpool")}
    paged.attention(s["q"], s["kpool"], s["vpool"], s["table"], s["cu"], s["ctx"], s["max_new"], out=s["out"])
    return {"out": s["out"]}


def _plain_plan(s):
    page = s["c"]["page"]
    ctx, new, held, table, free, count = (s[k].long() for k in ("ctx", "new", "held", "table", "free", "count"))
    B, max_pages = table.shape
    at = torch.arange(free.numel(), device=DEV)
    want = (ctx + new + page - 1) // page
    grow, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
    grow_end, back_end = grow.cumsum(0), back.cumsum(0)
    # the pages given back, in the order of requests, on top of the stack of free pages
    row = torch.searchsorted(back_end, at, right=True).clamp(max=B - 1)
    col = (want[row] + at - (back_end - back)[row]).clamp(0, max_pages - 1)
    given = table[row, col]
    stack = torch.where(at < count, free, given[(at - count).clamp(min=0)])
    top = count + back_end[-1]
    left = top - grow_end[-1]
    # the pages taken from its top
    row = torch.searchsorted(grow_end, at, right=True).clamp(max=B - 1)
    taken = stack[(top - 1 - at).clamp(0, free.numel() - 1)]
    col = held[row] + at - (grow_end - grow)[row]
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[torch.where(at < grow_end[-1], row * max_pages + col, flat.numel() - 1)] = taken
    table = flat[:-1].view(B, max_pages)
    # positions and slots of the new tokens
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    i = torch.arange(s["positions"].numel(), device=DEV)
    row = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
    pos = ctx[row] + i - cu[row]
    slot = table[row, (pos // page).clamp(max=max_pages - 1)] * page + pos % page
    live = i < cu[-1]
    minus = torch.full_like(pos, -1)
    out = {"table": table, "free": torch.where((at >= count) & (at < left), stack, free), "held_out": want,
           "count_out": left, "cu": cu, "positions": torch.where(live, pos, minus), "slots": torch.where(live, slot, minus)}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_norm_rope(s):
    c, n = s["c"], s["n"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    x = s["qkv"][:n].float().view(n, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if c["norm"]:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_gamma"].float()
        k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_gamma"].float()
    half = torch.arange(D // 2, device=DEV, dtype=torch.float64)
    angle = s["positions"][:n].double()[:, None] * THETA ** (-2.0 * half / D)  # far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    turn = lambda y: torch.cat([y[..., :D // 2] * cos - y[..., D // 2:] * sin,  # noqa: E731
                                y[..., D // 2:] * cos + y[..., :D // 2] * sin], -1)
    s["q"][:n] = turn(q).to(torch.bfloat16)
    slot = s["slots"][:n].long()
    s["kpool"][slot // page, :, slot % page] = turn(k).to(torch.bfloat16)
    s["vpool"][slot // page, :, slot % page] = v.to(torch.bfloat16)
    return {k: s[k] for k in ("q", "kpool", "vpool")}


def _plain_attention(s):
    c = s["c"]
    Hq, Hkv, D, page, B = c["Hq"], c["Hkv"], c["D"], c["page"], c["B"]
    T, L = s["max_new"], s["far"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    j, t = torch.arange(L, device=DEV), torch.arange(T, device=DEV)
    ids = s["table"].long().clamp(min=0)[:, j // page]  # [B, L]
    keys = s["kpool"][ids, :, j % page].float()  # [B, L, Hkv, D]
    values = s["vpool"][ids, :, j % page].float()
    rows = (cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, T, Hkv, Hq // Hkv, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, Hq // Hkv * T, D)
    score = torch.matmul(q, keys.permute(0, 2, 3, 1)) * D ** -0.5  # [B, Hkv, G T, L]
    score = score.view(B, Hkv, Hq // Hkv, T, L)
    hidden = j > (ctx[:, None] + t)[..., None]  # [B, T, L]
    score.masked_fill_(hidden[:, None, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    del score
    total = p.sum(-1)
    o = torch.matmul(p.view(B, Hkv, Hq // Hkv * T, L), values.permute(0, 2, 1, 3))
    o = o.view(B, Hkv, Hq // Hkv, T, D) / total[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, D).to(torch.bfloat16)
    # each new token's row of the padded batch, back in its place; rows behind the last sequence stay
    i = torch.arange(s["out"].shape[0], device=DEV)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
    at = (b * T + i - cu[b]).clamp(max=B * T - 1)
    s["out"].copy_(torch.where((i < cu[-1])[:, None, None], o[at], s["out"]))
    return {"out": s["out"]}


def _plain_verify(s):
    c = s["c"]
    B, K, V = c["B"], c["K"], c["V"]
    p, u, tok, length = s["p"], s["u"].double(), s["drafts"].long(), s["length"].long()
    b, t = torch.arange(B, device=DEV), torch.arange(K, device=DEV)
    target = p[b[:, None], t, tok].double()
    draft = s["q"][b[:, None], t, tok].double() if c["q"] else torch.ones_like(target)
    yes = (t < length[:, None]) & (u[:, :K] * draft < target)
    a = yes.long().cumprod(-1).sum(-1)
    # the last token: from what the target has over the draft, or, after the last draft, from the target itself;
    # in 64 bits, since a sum of 128256 values is compared with a number between its terms
    row = p[b, a].double()
    last = a.clamp(max=K - 1)
    if c["q"]:
        less = s["q"][b, last].double()
    else:
        less = (torch.arange(V, device=DEV) == tok[b, last][:, None]).double()
    rest = (row - less).clamp(min=0)
    rest = torch.where((a < length)[:, None] & (rest.sum(-1, keepdim=True) > 0), rest, row)
    cum = rest.cumsum(-1)
    pick = (cum <= u[b, K, None] * cum[:, -1:]).sum(-1).clamp(max=V - 1)
    i = torch.arange(K + 1, device=DEV)
    tokens = torch.where(i < a[:, None], torch.cat([tok, tok[:, :1]], -1), torch.full_like(i, -1))
    tokens = torch.where(i == a[:, None], pick[:, None], tokens)
    return {"tokens": tokens.to(torch.int32), "accepted": a.to(torch.int32)}


# ----------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": lambda _: None, "norm_rope": _exact_norm_rope, "attention": _exact_attention,
            "verify": lambda _: None}[case["op"]](s)


def _exact_norm_rope(s):
    c, n = s["c"], s["n"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    q, kpool, vpool = s["q"].double(), s["kpool"].double(), s["vpool"].double()
    x = s["qkv"][:n].double()
    pos, slot = s["positions"][:n].double(), s["slots"][:n].long()
    freq = torch.tensor([THETA ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64, device=DEV)
    spin = torch.polar(torch.ones(n, D // 2, dtype=torch.float64, device=DEV), pos[:, None] * freq)
    for h in range(Hq + 2 * Hkv):
        y = x[:, h * D:(h + 1) * D]
        if h < Hq + Hkv:
            if c["norm"]:
                y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
                y = y * (s["q_gamma"] if h < Hq else s["k_gamma"]).double()
            z = torch.complex(y[:, :D // 2].contiguous(), y[:, D // 2:].contiguous()) * spin
            y = torch.cat([z.real, z.imag], -1)
        if h < Hq:
            q[:n, h] = y
        else:
            pool = kpool if h < Hq + Hkv else vpool
            pool[slot // page, (h - Hq) % Hkv, slot % page] = y
    return {"q": q, "kpool": kpool, "vpool": vpool}


def _exact_attention(s):
    c = s["c"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    ctx, new = _lengths(c)
    out = s["out"].double()
    first = 0
    for b in range(c["B"]):
        n, L = new[b], ctx[b] + new[b]
        if not n:
            continue
        ids = s["table"][b, : _pages(L, page)].long()
        q = s["q"][first:first + n].double()
        see = torch.arange(L, device=DEV)[None] <= ctx[b] + torch.arange(n, device=DEV)[:, None]
        for g in range(Hkv):
            k = s["kpool"][ids, g].reshape(-1, D)[:L].double()
            v = s["vpool"][ids, g].reshape(-1, D)[:L].double()
            for h in range(g * G, (g + 1) * G):
                score = (q[:, h] @ k.T) / D ** 0.5
                out[first:first + n, h] = torch.softmax(score.masked_fill(~see, float("-inf")), -1) @ v
        first += n
    return {"out": out}
