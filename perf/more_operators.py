"""A paged cache held in 8 bits, and log probabilities of given tokens, as they are measured.

A serving step over a cache in 8 bits is, per layer: ``append`` (norms of
queries and keys for each head, the position rotation, and the stores of keys
and values as e4m3 with one scale for each page and head), then ``attention``
of the new tokens over those pages; and at the end ``logprobs``, what a server
answers with beside the tokens: each given token's log probability, the
entropy, and the likeliest alternatives.

The scale of a page and head is the smallest power of two s with max |x| <= 448 s
over the page's tokens: a page's first token sets it, a later token may raise
it, and then what the page holds is rounded to the larger scale.

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
E4M3 = torch.float8_e4m3fn


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one request, from the decoder's f32 activations
        dict(name="append_token", op="append", B=1, ctx_lo=4000, ctx_hi=4096, new_lo=1, new_hi=1, pad=0, Hq=32, Hkv=8,
             D=128, page=64, dtype="f32", norm=True, lens=1),
        # a decode batch, each request's token into a page that is partly filled
        dict(name="append_decode", op="append", B=64, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=1, pad=0, Hq=32, Hkv=8,
             D=128, page=16, dtype="bf16", norm=False, lens=2),
        # ragged chunks far into long contexts, a padded batch, seven query heads per key head, f32
        dict(name="append_chunks", op="append", B=5, ctx_lo=0, ctx_hi=1000000, new_lo=1, new_hi=300, pad=23, Hq=28,
             Hkv=4, D=128, page=32, dtype="f32", norm=True, lens=3),
        # a whole prompt from 16-bit activations
        dict(name="append_prompt", op="append", B=1, ctx_lo=0, ctx_hi=0, new_lo=8192, new_hi=8192, pad=0, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16", norm=True, lens=4),
        # the single token of the 8B-shaped decode workload, KV 4096
        dict(name="attention_token", op="attention", B=1, ctx_lo=4096, ctx_hi=4096, new_lo=1, new_hi=1, Hq=32, Hkv=8,
             D=128, page=64, pad=0, lens=1),
        # a decode batch over ragged lengths, small pages
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
        # one sampled token with the alternatives that a client asked for
        dict(name="logprobs_one", op="logprobs", N=1, V=128256, dtype="f32", top=5, masked=False),
        # a decode batch under constraints: most of the vocabulary is masked for some rows
        dict(name="logprobs_batch", op="logprobs", N=61, V=128256, dtype="f32", top=20, masked=True),
        # a prompt is scored, from 16-bit logits
        dict(name="logprobs_prompt", op="logprobs", N=2048, V=128256, dtype="bf16", top=1, masked=False),
    ]


HEADS = [(32, 8, 128), (28, 4, 128), (40, 8, 128), (8, 1, 128), (64, 8, 128), (4, 2, 64), (32, 4, 64), (12, 12, 64)]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random() + rng.random())))


def _draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "logprobs", "logprobs"])
    lens = rng.randrange(1 << 20)
    if op == "logprobs":
        return dict(op=op, N=_log(rng, 1, 2048), V=_log(rng, 1000, 128256), dtype=rng.choice(["f32", "bf16"]),
                    top=rng.choice([0, 1, 5, 20, rng.randrange(1, 33)]), masked=rng.random() < 0.25)
    page = rng.choice([16, 32, 64, 128])
    pad = rng.choice([0, 0, rng.randrange(1, 65)])
    Hq, Hkv, D = rng.choice(HEADS)
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
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=page, pad=pad, lens=lens, **shape)
    if op == "append":
        c.update(dtype=rng.choice(["f32", "bf16"]), norm=rng.random() < 0.75)
    return c


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("append", "attention", "logprobs")}
    while True:
        c = _draw(rng)
        if _cost(c) > most[c["op"]]:
            continue
        if c["op"] != "logprobs":
            ctx, new = _lengths(c)
            if max(new) < 1:
                continue
            far = max(a + b for a, b in zip(ctx, new))
            # the plain form holds every score of a padded batch
            if c["op"] == "attention" and (c["B"] * c["Hq"] * max(new) * far > 1 << 31 or
                                           c["B"] * c["Hkv"] * c["D"] * far > 1 << 30):
                continue
        return c


def _lengths(c):
    """(cached tokens, new tokens) of every request: the case's own, whatever the seed."""
    r = random.Random(c["lens"])
    return ([r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["B"])],
            [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])])


def _pages(n, page):
    return -(-n // page)


def work(case):
    c = case
    if c["op"] == "logprobs":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["N"] * (c["V"] * size + 12 + 8 * c["top"]), "flops": 6 * c["N"] * c["V"]}
    ctx, new = _lengths(c)
    n = sum(new)
    if c["op"] == "append":
        size = 4 if c["dtype"] == "f32" else 2
        touched = sum(_pages(a + b, c["page"]) - a // c["page"] for a, b in zip(ctx, new) if b)
        begun = sum(1 for a, b in zip(ctx, new) if b and a % c["page"])  # pages with a scale already
        return {"bytes": n * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * size + n * (2 * c["Hq"] + 2 * c["Hkv"]) * c["D"]
                + 8 * (n + c["pad"]) + 4 * c["D"] + 8 * c["Hkv"] * (touched + begun),
                "flops": n * ((c["Hq"] + c["Hkv"]) * c["D"] * (7 if c["norm"] else 3) + 4 * c["Hkv"] * c["D"])}
    keys = sum(a + b for a, b in zip(ctx, new) if b)
    pages = sum(_pages(a + b, c["page"]) for a, b in zip(ctx, new) if b)
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, new))
    return {"bytes": keys * c["Hkv"] * c["D"] * 2 + pages * (8 * c["Hkv"] + 4) + n * c["Hq"] * c["D"] * 4 + 8 * c["B"],
            "flops": 4 * c["D"] * c["Hq"] * pairs}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    return {"append": _prepare_append, "attention": _prepare_attention, "logprobs": _prepare_logprobs}[case["op"]](
        case, seed)


def _pow2_scale(amax):
    """The smallest power of two s (2^-126 at least) with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.full_like(e, -126)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), e)


def _filled(num_pages, Hkv, page, D, g, spread):
    """A pool whose pages hold values of different magnitude, and the scales: keys and values as a model has them,
    about one in size, some pages larger than others."""
    x = torch.randn(num_pages, Hkv, page, D, generator=g, device=DEV, dtype=torch.bfloat16)
    x *= torch.exp2(spread * torch.randn(num_pages, Hkv, 1, 1, generator=g, device=DEV)).to(torch.bfloat16)
    scale = _pow2_scale(x.abs().amax((2, 3)).float())
    return (x * (1 / scale).to(torch.bfloat16)[:, :, None, None]).to(E4M3), scale


def _prepare_append(c, seed):
    g = _gen(seed)
    ctx, new = _lengths(c)
    n, page = sum(new), c["page"]
    rows = n + c["pad"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    qkv = torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
    gain = [(1 + 0.02 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
            for _ in range(2)]
    # the pages that the new tokens go to, anywhere in the pool
    pages = [_pages(a + b, page) - a // page if b else 0 for a, b in zip(ctx, new)]
    num_pages = sum(pages) + 3
    ids = torch.randperm(num_pages, generator=g, device=DEV)
    first = [0]
    for k in pages:
        first.append(first[-1] + k)
    count = _i32(new).long()
    b = torch.repeat_interleave(torch.arange(c["B"], device=DEV), count)
    pos = _i32(ctx).long()[b] + torch.arange(n, device=DEV) - (count.cumsum(0) - count)[b]
    at = ids[_i32(first).long()[b] + pos // page - (_i32(ctx).long() // page)[b]]
    slots = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    positions = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    slots[:n] = (at * page + pos % page).to(torch.int32)
    positions[:n] = pos.to(torch.int32)
    kpool, kscale = _filled(num_pages, Hkv, page, D, g, 0.7)
    vpool, vscale = _filled(num_pages, Hkv, page, D, g, 0.7)
    return dict(c=c, qkv=qkv, q_gamma=gain[0], k_gamma=gain[1], positions=positions, slots=slots, kpool=kpool,
                vpool=vpool, kscale=kscale, vscale=vscale,
                q=torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=DEV), n=n)


def _prepare_attention(c, seed):
    g = _gen(seed)
    ctx, new = _lengths(c)
    n, D, page = sum(new), c["D"], c["page"]
    pages = [_pages(a + b, page) for a, b in zip(ctx, new)]
    num_pages, max_pages = sum(pages) + 5, max(pages) + 1
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["B"], max_pages), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max_pages, device=DEV)[None, :] < _i32(pages)[:, None]] = ids[: sum(pages)]
    kpool, kscale = _filled(num_pages, c["Hkv"], page, D, g, 0.25)
    vpool, vscale = _filled(num_pages, c["Hkv"], page, D, g, 0.5)
    q = torch.randn(n + c["pad"], c["Hq"], D, generator=g, device=DEV) * 1.5
    cu = [0]
    for b in new:
        cu.append(cu[-1] + b)
    return dict(c=c, q=q.to(torch.bfloat16), kpool=kpool, vpool=vpool, kscale=kscale, vscale=vscale, table=table,
                cu=_i32(cu), ctx=_i32(ctx), max_new=max(new), far=max(a + b for a, b in zip(ctx, new)),
                out=torch.zeros(n + c["pad"], c["Hq"], D, dtype=torch.bfloat16, device=DEV))


def _prepare_logprobs(c, seed):
    g = _gen(seed)
    N, V = c["N"], c["V"]
    logits = torch.randn(N, V, generator=g, device=DEV) * 2.5
    tokens = torch.randint(0, V, (N,), generator=g, device=DEV)
    # tokens of a text are mostly among the likely ones
    logits[torch.arange(N, device=DEV), tokens] += 9 * torch.rand(N, generator=g, device=DEV)
    if c["masked"]:  # every other row is constrained to a few hundred tokens, the given one among them
        few = torch.rand(N, V, generator=g, device=DEV) > 300 / V
        few[::2] = False
        few[torch.arange(N, device=DEV), tokens] = False
        logits.masked_fill_(few, float("-inf"))
    return dict(c=c, logits=logits if c["dtype"] == "f32" else logits.to(torch.bfloat16), tokens=tokens.to(torch.int32))


# ----------------------------------------------------------------- one pass
def run(state):
    op = state["c"]["op"]
    if own:
        return _own(op, state)
    return {"append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs}[op](state)


def _own(op, s):
    c = s["c"]
    if op == "logprobs":
        from task_graph_interpreter_gb300 import logprobs
        r = logprobs.token_logprobs(s["logits"], s["tokens"], top=c["top"])
        out = {"logprobs": r.logprobs, "entropy": r.entropy}
        return dict(out, top_ids=r.top_ids, top_logprobs=r.top_logprobs) if c["top"] else out
    from task_graph_interpreter_gb300 import paged
    if op == "append":
        paged.qk_norm_rope(s["qkv"], c["Hq"], c["Hkv"], c["D"], s["positions"], s["slots"], s["kpool"], s["vpool"],
                           kscale=s["kscale"], vscale=s["vscale"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=EPS,
                           rope_theta=THETA, out=s["q"])
        return {k: s[k] for k in ("q", "kpool", "vpool", "kscale", "vscale")}
    paged.attention(s["q"], s["kpool"], s["vpool"], s["table"], s["cu"], s["ctx"], s["max_new"], kscale=s["kscale"],
                    vscale=s["vscale"], out=s["out"])
    return {"out": s["out"]}


def _plain_append(s):
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
    _plain_store(s["kpool"], s["kscale"], slot // page, slot % page, turn(k))
    _plain_store(s["vpool"], s["vscale"], slot // page, slot % page, v)
    return {k: s[k] for k in ("q", "kpool", "vpool", "kscale", "vscale")}


def _plain_store(pool, scale, at, off, x):
    """Rows x [n, Hkv, D] to pages `at`, offsets `off`: scales of the touched pages, what they hold rounded to a scale
    that grew, and the rows."""
    num_pages, Hkv, page, D = pool.shape
    amax = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(-1), "amax")
    first = torch.full((num_pages,), page, device=DEV).index_reduce_(0, at, off, "amin")
    need = _pow2_scale(amax)
    grown = torch.where((first > 0)[:, None], torch.maximum(need, scale), need)
    grown = torch.where((first < page)[:, None], grown, scale)
    codes = pool.view(torch.uint8)
    held = (torch.arange(page, device=DEV) < first[:, None]) & (first < page)[:, None]
    held = held[:, None] & (grown != scale)[..., None]
    again = (pool.float() * (scale / grown)[..., None, None]).to(E4M3).view(torch.uint8)
    codes.copy_(torch.where(held[..., None], again, codes))
    codes[at, :, off] = (x / grown[at][..., None]).to(E4M3).view(torch.uint8)
    scale.copy_(grown)


def _plain_attention(s):
    c = s["c"]
    Hq, Hkv, D, page, B = c["Hq"], c["Hkv"], c["D"], c["page"], c["B"]
    T, L = s["max_new"], s["far"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    j, t = torch.arange(L, device=DEV), torch.arange(T, device=DEV)
    ids = s["table"].long().clamp(min=0)[:, j // page]  # [B, L]
    # codes and their scales: [B, L, Hkv, D]
    keys = s["kpool"].view(torch.uint8)[ids, :, j % page].view(E4M3).float() * s["kscale"][ids][..., None]
    values = s["vpool"].view(torch.uint8)[ids, :, j % page].view(E4M3).float() * s["vscale"][ids][..., None]
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
    values = values * (j < (ctx + cu[1:] - cu[:-1])[:, None])[..., None, None]  # nothing of other requests' pages
    o = torch.matmul(p.view(B, Hkv, Hq // Hkv * T, L), values.permute(0, 2, 1, 3))
    o = o.view(B, Hkv, Hq // Hkv, T, D) / total[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, D).to(torch.bfloat16)
    # each new token's row of the padded batch, back in its place; rows behind the last sequence stay
    i = torch.arange(s["out"].shape[0], device=DEV)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
    at = (b * T + i - cu[b]).clamp(max=B * T - 1)
    s["out"].copy_(torch.where((i < cu[-1])[:, None, None], o[at], s["out"]))
    return {"out": s["out"]}


def _plain_logprobs(s):
    top = s["c"]["top"]
    x = s["logits"].float()
    y = x - x.amax(-1, keepdim=True)
    e = torch.exp(y)
    total = e.sum(-1, keepdim=True)
    lp = y - torch.log(total)
    out = {"logprobs": lp.gather(-1, s["tokens"].long()[:, None])[:, 0],
           "entropy": torch.log(total[:, 0]) - (e * y.clamp(min=-1e30)).sum(-1) / total[:, 0]}
    if not top:
        return out
    # a stable order: of equal ones the lowest index first
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    return dict(out, top_ids=ids.to(torch.int32), top_logprobs=lp.gather(-1, ids))


# ----------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_append(s):
    c, n = s["c"], s["n"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    x = s["qkv"][:n].double()
    pos, slot = s["positions"][:n].double(), s["slots"][:n].long()
    freq = torch.tensor([THETA ** (-2 * i / D) for i in range(D // 2)], dtype=torch.float64, device=DEV)
    spin = torch.polar(torch.ones(n, D // 2, dtype=torch.float64, device=DEV), pos[:, None] * freq)
    out = {"q": s["q"].double(), "kpool": s["kpool"].double(), "vpool": s["vpool"].double(),
           "kscale": s["kscale"].double(), "vscale": s["vscale"].double()}
    order = torch.argsort(slot)
    at, rank = torch.unique(slot[order] // page, return_inverse=True)  # the touched pages
    off = slot[order] % page
    for h in range(Hq + 2 * Hkv):
        y = x[:, h * D:(h + 1) * D]
        if h < Hq + Hkv:
            if c["norm"]:
                y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
                y = y * (s["q_gamma"] if h < Hq else s["k_gamma"]).double()
            z = torch.complex(y[:, :D // 2].contiguous(), y[:, D // 2:].contiguous()) * spin
            y = torch.cat([z.real, z.imag], -1)
        if h < Hq:
            out["q"][:n, h] = y
            continue
        g, name = (h - Hq) % Hkv, "k" if h < Hq + Hkv else "v"
        pool, scale = out[name + "pool"], out[name + "scale"]
        y = y[order]
        # every touched page in full: what it holds below the first new row, then the new rows
        new = torch.zeros(len(at), page, D, dtype=torch.float64, device=DEV)
        new[rank, off] = y
        live = torch.zeros(len(at), page, dtype=torch.bool, device=DEV)
        live[rank, off] = True
        begun = ~live[:, 0]
        top = new.abs().flatten(1).max(1).values
        want = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-126))
        old = scale[at, g]
        now = torch.where(begun & (old > want), old, want)
        below = live.cumsum(1) == 0
        codes = pool[at, g]
        again = _e4m3(codes * (old / now)[:, None, None])
        codes = torch.where(below[..., None] & (now != old)[:, None, None], again, codes)
        pool[at, g] = torch.where(live[..., None], _e4m3(new / now[:, None, None]), codes)
        scale[at, g] = now
    return out


def _e4m3(x):
    """64-bit values rounded to e4m3: four significant bits, steps of 2^-9 at least, ties to even."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448, 448)


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
            k, v = ((s[w + "pool"][:, g].view(torch.uint8)[ids].view(E4M3).double()
                     * s[w + "scale"][ids, g].double()[:, None, None]).reshape(-1, D)[:L] for w in "kv")
            for h in range(g * G, (g + 1) * G):
                score = (q[:, h] @ k.T) / D ** 0.5
                out[first:first + n, h] = torch.softmax(score.masked_fill(~see, float("-inf")), -1) @ v
        first += n
    return {"out": out}


def _exact_logprobs(s):
    top, N = s["c"]["top"], s["c"]["N"]
    parts = []
    for i in range(0, N, 256):
        x = s["logits"][i:i + 256].double()
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        p = torch.exp(lp)
        one = {"logprobs": lp[torch.arange(len(x), device=DEV), s["tokens"][i:i + 256].long()],
               "entropy": -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)}
        if top:
            one["top_logprobs"] = torch.topk(lp, top, dim=-1).values
        parts.append(one)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return dict(out, top_ids=None) if top else out
