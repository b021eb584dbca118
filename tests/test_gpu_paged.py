"""The paged-cache operators against plain float64 implementations: the step
plan, the per-head norms with rotation and page stores, attention of new
tokens over the pages, and a run of them together.

Tolerances count roundings.  A bf16 result is off by 2^-8 of its value (half
a step, eps / 2).  Attention adds what the probabilities lose: with
A = sum_j w_j |v_j| (w the softmax weights), a relative error e of every
weight moves the result by at most 2 e A (numerator and sum).  e is 2^-8 where
the chunk kernel rounds probabilities to bf16, 2^-16 where the few-rows kernel
splits them in two parts, plus the scores' own error: D terms summed in f32
(each partial sum off by at most 2^-23 of it, tensor cores truncate) and the
exponent's 2^-23 relative error, both times |score| sums.
"""
import math

import numpy as np
import pytest
import torch

from task_graph_interpreter_gb300 import _lib as L
from task_graph_interpreter_gb300 import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plan
def plan_ref(ctx, new, table, held, free, page):
    """Lists in, lists out; the operator's definition, page by page."""
    table, free = [list(r) for r in table], list(free)
    want = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    for b, w in enumerate(want):
        free += table[b][w:held[b]]
    for b, w in enumerate(want):
        for j in range(held[b], w):
            table[b][j] = free.pop()
    pos, slots, cu = [], [], [0]
    for b, n in enumerate(new):
        for t in range(n):
            p = ctx[b] + t
            pos.append(p)
            slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
    return table, want, free, cu, pos, slots


def plan_case(B, page, ctx_hi, new_hi, seed, spare=7):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, B).tolist()
    new = rng.integers(0, new_hi + 1, B).tolist()
    held = [-(-c // page) + int(rng.integers(0, 3)) for c in ctx]
    for b in range(0, B, 5):  # finished requests
        ctx[b] = new[b] = 0
    want = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    grow = sum(max(0, w - h) for w, h in zip(want, held))
    pages = sum(held) + max(0, grow) + spare
    ids = rng.permutation(pages).tolist()
    width = max(max(held), max(want)) + 1
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    return ctx, new, table, held, ids[at:], pages


def run_plan(ctx, new, table, held, free, pages, page, max_tokens, in_place=True, offset=0):
    t = dict(table=i32(table), held=i32(held), free=i32(free + [-7] * (pages - len(free))), count=i32([len(free)]),
             status=i32([0]), ho=i32([-9] * len(held)), co=i32([-9]))
    pos = i32([-5] * (max_tokens + offset))[offset:]
    slots = i32([-5] * (max_tokens + offset))[offset:]
    out = {} if in_place else dict(held_out=t["ho"], count_out=t["co"])
    pl = paged.plan(i32(ctx), i32(new), t["table"], t["held"], t["free"], t["count"], page, positions=pos, slots=slots,
                    status=t["status"], **out)
    h, c = (t["held"], t["count"]) if in_place else (t["ho"], t["co"])
    return t, pl.cu.tolist(), pos.tolist(), slots.tolist(), h.tolist(), int(c), int(t["status"])


@pytest.mark.parametrize("B,page,ctx_hi,new_hi,pad,in_place,offset", [
    (1, 16, 0, 1, 0, True, 0), (1, 64, 100, 5, 3, False, 1), (7, 16, 200, 30, 5, True, 0), (33, 32, 500, 1, 0, False, 0),
    (600, 16, 300, 40, 2, True, 0), (513, 128, 300, 40, 1, False, 3), (4096, 16, 60, 3, 11, True, 0),
    (3, 256, 9000, 5000, 0, True, 0)])
def test_plan_matches_its_definition(B, page, ctx_hi, new_hi, pad, in_place, offset):
    ctx, new, table, held, free, pages = plan_case(B, page, ctx_hi, new_hi, B * 31 + page)
    n = sum(new)
    want = plan_ref(ctx, new, table, held, free, page)
    t, cu, pos, slots, h, c, status = run_plan(ctx, new, table, held, free, pages, page, max(1, n + pad), in_place,
                                               offset)
    assert status == 0
    assert t["table"].tolist() == want[0] and h == want[1] and cu == want[3]
    assert c == len(want[2]) and t["free"].tolist()[:c] == want[2]
    pad = max(1, n + pad) - n
    assert pos == want[4] + [-1] * pad and slots == want[5] + [-1] * pad
    if not in_place:
        assert t["held"].tolist() == held and int(t["count"]) == len(free)


@pytest.mark.parametrize("what,code", [("pages", L.MK_DEV_CAPACITY), ("tokens", L.MK_DEV_CAPACITY),
                                       ("width", L.MK_DEV_CAPACITY), ("negative", L.MK_DEV_BAD_INDEX),
                                       ("held", L.MK_DEV_BAD_INDEX), ("count", L.MK_DEV_BAD_INDEX)])
def test_plan_that_does_not_fit_moves_nothing(what, code):
    ctx, new, table, held, free, pages = plan_case(20, 16, 100, 30, 3)
    n = sum(new)
    if what == "pages":  # the pages that go back and the free ones are one too few
        want = [-(-(c + k) // 16) for c, k in zip(ctx, new)]
        new[1] += 16 * (1 + sum(h - w for h, w in zip(held, want)) + len(free))
        table = [r + [-1] * (new[1] // 16 + 1) for r in table]
        n = sum(new)
    if what == "width":
        ctx[1] = 16 * len(table[0]) + 1
    if what == "negative":
        new[2] = -1
    if what == "held":
        held[3] = len(table[0]) + 1
    if what == "count":
        pages = len(free) - 1
    free_in = free + [-7] * max(0, pages - len(free))
    t = dict(table=i32(table), held=i32(held), free=i32(free_in[:pages]), count=i32([len(free)]), status=i32([0]))
    m = n - 1 if what == "tokens" else n + 4
    pl = paged.plan(i32(ctx), i32(new), t["table"], t["held"], t["free"], t["count"], 16, max_tokens=m,
                    status=t["status"])
    assert int(t["status"]) == code
    assert t["table"].tolist() == table and t["held"].tolist() == held and int(t["count"]) == len(free)
    assert t["free"].tolist() == free_in[:pages]
    assert pl.cu.tolist() == [0] * 21 and pl.positions.tolist() == [-1] * m and pl.slots.tolist() == [-1] * m


def test_plan_reports_a_page_outside_the_pool():
    # the first request's page is not in the pool, the second takes one off the stack that is not
    t = dict(table=i32([[99, -1], [-1, -1]]), held=i32([1, 0]), free=i32([0, 1, 50, -1]), count=i32([3]), status=i32([0]))
    pl = paged.plan(i32([3, 0]), i32([2, 1]), t["table"], t["held"], t["free"], t["count"], 16, max_tokens=4,
                    status=t["status"])
    assert int(t["status"]) == L.MK_DEV_BAD_INDEX
    assert pl.positions.tolist() == [3, 4, 0, -1] and pl.slots.tolist() == [-1] * 4
    assert t["table"].tolist() == [[99, -1], [50, -1]]


# ------------------------------------------------------------------ norms, rotation, stores
def norm_rope_ref(x, gamma, pos, eps, theta):
    """x float64 [N, D] -> normed (gamma given) and turned, and the size its f32 errors scale with."""
    D = x.shape[-1]
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    ang = pos[:, None].astype(np.float64) * theta ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[:, :D // 2], x[:, D // 2:]
    size = np.abs(a) + np.abs(b)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), np.concatenate([size, size], -1)


@pytest.mark.parametrize("N,Hq,Hkv,D,dtype,norm,far,page,strided", [
    (1, 32, 8, 128, torch.float32, "both", 0, 64, False), (5, 4, 2, 64, torch.float32, "none", 100, 16, True),
    (37, 28, 4, 128, torch.bfloat16, "both", 1000000, 16, True), (130, 8, 1, 128, torch.float32, "q", 2 ** 31 - 1000, 32, False),
    (77, 12, 12, 64, torch.bfloat16, "k", 5000, 256, False), (700, 3, 1, 64, torch.float32, "both", 70000, 128, True),
    (2100, 32, 8, 128, torch.bfloat16, "none", 8000, 64, False)])
def test_norm_rope_matches_float64(N, Hq, Hkv, D, dtype, norm, far, page, strided):
    g = torch.Generator(device=DEV).manual_seed(N)
    width, theta, eps = (Hq + 2 * Hkv) * D, 5e5, 1e-5
    qkv = torch.randn(N, width + (24 if strided else 0), device=DEV, generator=g).to(dtype)[:, :width]
    gq = (1 + 0.1 * torch.randn(D, device=DEV, generator=g)).bfloat16() if norm in ("both", "q") else None
    gk = (1 + 0.1 * torch.randn(D, device=DEV, generator=g)).bfloat16() if norm in ("both", "k") else None
    pages = -(-N // page) + 2
    perm = torch.randperm(pages * page, device=DEV, generator=g)[:N].int()
    pos = far + torch.arange(N, device=DEV, dtype=torch.int32)
    slots = perm.clone()
    out = torch.full((N, Hq + 1, D), 7.0, dtype=torch.bfloat16, device=DEV)[:, :Hq]
    pool = [torch.full((pages, Hkv, page, D), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    status = i32([0])
    left_out = not_stored = None
    if N > 4:
        left_out, not_stored = 2, 3
        pos[left_out] = -1
        slots[not_stored] = -1
    paged.qk_norm_rope(qkv, Hq, Hkv, D, pos, slots, pool[0], pool[1], q_gamma=gq, k_gamma=gk, eps=eps, rope_theta=theta,
                       out=out, status=status)
    assert int(status) == 0
    x = qkv.double().cpu().numpy().reshape(N, Hq + 2 * Hkv, D)
    p = pos.cpu().numpy().astype(np.int64)
    got_q = out.double().cpu().numpy()
    flat = [t.permute(0, 2, 1, 3).reshape(pages * page, Hkv, D).double().cpu().numpy() for t in pool]
    sl = slots.cpu().numpy()
    rows = np.array([r for r in range(N) if r != left_out])
    stored = np.array([r for r in rows if r != not_stored])
    # a bf16 result (2^-8 of it), and f32 arithmetic before it: the mean (D + 3 roundings), the root,
    # four products and the angle's 2^-23, all under 2^-17 of the pair's size
    def check(got, x, gamma, pos):
        want, size = norm_rope_ref(x, None if gamma is None else gamma.double().cpu().numpy(), pos, eps, theta)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * size + 1e-30
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)
    for h in range(Hq):
        check(got_q[rows, h], x[rows, h], gq, p[rows])
    for h in range(Hkv):
        check(flat[0][sl[stored], h], x[stored, Hq + h], gk, p[stored])
        assert np.all(np.abs(flat[1][sl[stored], h] - x[stored, Hq + Hkv + h])
                      <= 2.0 ** -8 * np.abs(x[stored, Hq + Hkv + h]))
    # everything else stays
    if left_out is not None:
        assert np.all(got_q[left_out] == 7.0)
    other = np.ones(pages * page, bool)
    other[sl[stored]] = False
    assert np.all(flat[0][other] == 3.0) and np.all(flat[1][other] == 3.0)


def test_norm_rope_reports_a_slot_outside_the_pool():
    qkv = torch.ones(3, 4 * 64, device=DEV)
    pool = [torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    status = i32([0])
    q = paged.qk_norm_rope(qkv, 2, 1, 64, i32([0, 0, 0]), i32([31, 32, 2 ** 31 - 1]), pool[0], pool[1], status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    assert torch.all(q == 1.0) and torch.all(pool[1][1, 0, 15] == 1.0)
    assert float(pool[0].abs().sum()) == 64.0 and float(pool[1].abs().sum()) == 64.0


# ------------------------------------------------------------------ attention
def attention_case(ctx, new, Hq, Hkv, D, page, seed, junk=True, spare=3):
    """A pool whose unused rows hold NaN, requests on scattered pages."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + spare
    ids = torch.randperm(pages, device=DEV, generator=g)
    width = max(need + [1]) + 1
    table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEV)
    pool = [torch.full((pages, Hkv, page, D), float("nan") if junk else 0.0, dtype=torch.bfloat16, device=DEV)
            for _ in range(2)]
    at = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        mine = ids[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine.int()
        for j in range(need[b]):
            rows = min(page, c + n - j * page)
            for t in pool:
                t[mine[j], :, :rows] = torch.randn(Hkv, rows, D, device=DEV, generator=g).bfloat16()
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (1.5 * torch.randn(cu[-1], Hq, D, device=DEV, generator=g)).bfloat16()
    return q, pool[0], pool[1], table, cu


def attention_ref(q, kpool, vpool, table, cu, ctx, page, scale, lost=()):
    """float64 (result, sum of weights times |v|, largest sum of |q||k|); `lost`: (request, page index) left out."""
    Hq, D = q.shape[1:]
    Hkv = kpool.shape[1]
    G = Hq // Hkv
    out, size = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    reach = 0.0
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        Lb = ctx[b] + n
        ids = table[b, : -(-Lb // page)].long().clamp(0, kpool.shape[0] - 1)
        k = kpool[ids].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :Lb].double()
        v = vpool[ids].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :Lb].double()
        j = torch.arange(Lb, device=DEV)
        see = j[None] <= ctx[b] + torch.arange(n, device=DEV)[:, None]
        for (rb, rj) in lost:
            if rb == b:
                see &= (j // page != rj)[None]
        qb = q[cu[b]:cu[b + 1]].double()
        for h in range(Hq):
            s = (qb[:, h] @ k[h // G].T * scale).masked_fill(~see, -math.inf)
            w = torch.nan_to_num(torch.softmax(s, -1))  # a row that sees no key is zero
            w = torch.where(see, w, 0.0)
            vv = torch.where(see.any(0)[:, None], v[h // G], 0.0)
            out[cu[b]:cu[b + 1], h] = w @ vv
            size[cu[b]:cu[b + 1], h] = w @ vv.abs()
            a = (qb[:, h].abs() @ k[h // G].abs().T * scale).masked_fill(~see, 0.0)
            reach = max(reach, float(torch.nan_to_num(a).max()))
    return out, size, reach


def is_few(new, Hq, Hkv):
    """Whether the few-rows kernel takes the call (the chunk kernel rounds probabilities to bf16)."""
    return max(new) * (Hq // Hkv) <= 8


def attention_close(got, want, size, reach, D, few):
    e = (2.0 ** -16 if few else 2.0 ** -8) + reach * (D + 4) * 2.0 ** -23
    tol = 2.0 ** -8 * want.abs() + 2 * e * size + 1e-30
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), f"max excess {float((err - tol).max())}, max error {float(err.max())}"


FEW = [  # ctx, new, Hq, Hkv, D, page
    ([0], [1], 4, 2, 64, 16), ([0], [1], 32, 8, 128, 64), ([1], [1], 8, 1, 128, 16), ([4096], [1], 32, 8, 128, 64),
    ([31, 32, 33, 63, 64, 65], [1] * 6, 32, 8, 128, 32), ([15, 16, 17, 127, 128, 129], [1] * 6, 12, 12, 64, 16),
    ([700, 0, 5, 3000, 12], [1, 0, 1, 1, 0], 28, 4, 128, 16), ([1000, 0, 77], [5, 8, 1], 16, 4, 128, 128),
    ([0, 3, 250], [8, 8, 3], 32, 8, 64, 256), ([333], [1], 32, 1, 64, 32), ([513, 100], [4, 2], 8, 1, 128, 16),
    ([513, 100], [4, 2], 4, 2, 128, 16), ([30, 31, 32, 33], [8, 7, 6, 5], 3, 3, 64, 16), ([100] * 300, [1] * 300, 4, 2, 64, 16), ([20000, 9], [1, 1], 40, 8, 128, 16)]
CHUNK = [
    ([0], [9], 4, 1, 64, 16), ([0], [128], 4, 4, 128, 64), ([0], [129], 12, 12, 64, 16), ([5, 0, 300], [40, 1, 77], 32, 8, 128, 32),
    ([0, 1000, 0, 64], [700, 33, 0, 256], 32, 4, 64, 16), ([100, 37], [257, 511], 28, 4, 128, 128),
    ([2000], [64], 8, 1, 128, 256), ([0], [1500], 5, 5, 128, 16), ([127, 128, 129], [127, 128, 129], 6, 2, 64, 64),
    ([50], [30], 96, 1, 64, 32), ([0] * 40, [33 + i for i in range(40)], 8, 2, 128, 16)]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", FEW)
def test_attention_of_tokens_and_drafts(ctx, new, Hq, Hkv, D, page):
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, len(ctx) + D)
    status = i32([0])
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), status=status)
    assert int(status) == 0
    attention_close(got, *attention_ref(q, k, v, table, cu, ctx, page, D ** -0.5), D, is_few(new, Hq, Hkv))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", CHUNK)
def test_attention_of_chunks(ctx, new, Hq, Hkv, D, page):
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, len(ctx) + D)
    status = i32([0])
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), status=status)
    assert int(status) == 0
    attention_close(got, *attention_ref(q, k, v, table, cu, ctx, page, D ** -0.5), D, False)


@pytest.mark.parametrize("new", [[2, 1, 2], [2, 1, 3], [60, 1, 33]])
def test_attention_strides_and_rows_of_no_request(new):
    """Queries inside a wider row, outputs apart, rows before, between and behind the requests' own; a scale."""
    ctx, Hq, Hkv, D, page = [40, 0, 500], 8, 2, 128, 16
    q0, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 11)
    n = cu[-1]
    wide = torch.full((n + 9, Hq + 4, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[3:3 + n, :Hq] = q0
    out = torch.full((n + 9, Hq + 2, D), 5.0, dtype=torch.bfloat16, device=DEV)
    got = paged.attention(wide[:, :Hq], k, v, table, i32([c + 3 for c in cu]), i32(ctx), max(new), out=out[:, :Hq],
                          scale=0.2)
    want, size, reach = attention_ref(q0, k, v, table, cu, ctx, page, 0.2)
    attention_close(got[3:3 + n], want, size, reach, D, is_few(new, Hq, Hkv))
    assert torch.all(out[:3] == 5.0) and torch.all(out[3 + n:] == 5.0) and torch.all(out[:, Hq:] == 5.0)


@pytest.mark.parametrize("new", [[1, 2, 1], [1, 1, 4], [50, 40, 3]])
def test_attention_leaves_out_pages_outside_the_pool(new):
    ctx, Hq, Hkv, D, page = [300, 10, 90], 16, 4, 128, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 12)
    keep = table.clone()
    table[0, 3] = -1
    table[0, 11] = k.shape[0]
    table[1] = 2 ** 31 - 1   # nothing of the second request is there
    status = i32([0])
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    lost = [(0, 3), (0, 11)] + [(1, j) for j in range(table.shape[1])]
    attention_close(got, *attention_ref(q, k, v, keep, cu, ctx, page, D ** -0.5, lost), D, is_few(new, Hq, Hkv))
    assert torch.all(got[cu[1]:cu[2]] == 0)


@pytest.mark.parametrize("new,few", [([1, 1], True), ([40, 20], False)])
@pytest.mark.parametrize("what", ["cu", "past", "max_new", "pages", "negative"])
def test_attention_refuses_lengths_that_do_not_fit(new, few, what):
    ctx, Hq, Hkv, D, page = [30, 40], 8, 2, 64, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 13)
    cu2, ctx2, most = list(cu), list(ctx), max(new)
    if what == "cu":
        cu2[1] = cu2[2] + 1
    elif what == "past":
        cu2[2] += 1
        most += 1
    elif what == "max_new":
        most = 40 if not few else 1
        cu2 = [0, cu[-1], cu[-1]]
        if not few:
            q = torch.cat([q, q])
            cu2 = [0, 41, 60]
    elif what == "pages":
        ctx2[0] = table.shape[1] * page
    else:
        ctx2[1] = -1
    out = torch.full_like(q, 5.0)
    status = i32([0])
    paged.attention(q, k, v, table, i32(cu2), i32(ctx2), most, out=out, status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    assert torch.all(out == 5.0)


@pytest.mark.parametrize("shift", [3e4, -3e4])
@pytest.mark.parametrize("new", [[2], [3], [70]])
def test_attention_with_far_apart_scores(new, shift):
    """Scores that jump by thousands from key to key (running maxima move, old sums vanish) and rows of equal scores."""
    ctx, Hq, Hkv, D, page = [400], 4, 1, 128, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 14)
    q.zero_()
    q[:, 0, 0] = 1.0
    q[:, 1, 0] = 64.0
    ids = table[0, : -(-(ctx[0] + new[0]) // page)].long()
    flat = torch.arange(ids.numel() * page, device=DEV, dtype=torch.float32)
    ramp = torch.round(flat / flat.numel() * 64) / 64 * shift   # bf16 steps
    k[ids, 0, :, 0] = ramp.view(-1, page).bfloat16()
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), scale=1.0)
    want, size, _ = attention_ref(q, k, v, table, cu, ctx, page, 1.0)
    # one product per score, exact in f32; the exponent's error is 2^-23 of the difference to the
    # maximum, which matters only where that is under 150 or so
    e = (2.0 ** -16 if is_few(new, Hq, Hkv) else 2.0 ** -8) + 150 * 2.0 ** -22
    assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * e * size + 1e-30).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("new", [[2], [8], [100]])
def test_attention_rows_before_a_bad_key_are_untouched(new, bad):
    """A key and value that are not finite reach the rows that see them, and no others."""
    ctx, Hq, Hkv, D, page = [37], 4, 1, 64, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 15)
    clean = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new))
    t = new[0] // 2
    at = ctx[0] + t
    v[int(table[0, at // page]), 0, at % page, 5] = bad
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new))
    assert torch.equal(got[:t], clean[:t])
    assert not torch.isfinite(got[t:, :, 5]).any()
    other = [d for d in range(D) if d != 5]
    assert torch.equal(got[t:][..., other], clean[t:][..., other])
    k[int(table[0, at // page]), 0, at % page, 3] = math.nan
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new))
    assert torch.equal(got[:t], clean[:t]) and torch.isnan(got[t:]).all()


# ------------------------------------------------------------------ together
def test_a_serving_loop_over_pages():
    """Prompts, then tokens, then drafts rolled back, on two layers: every step's attention against
    float64 over a contiguous history; requests end and their pages are used again; the same on another
    stream and replayed from a CUDA graph."""
    Hq, Hkv, D, page, layers, R = 8, 2, 64, 16, 2, 3
    c = paged.PagedCache(layers, 24, page, Hkv, D, R, 16, 96)
    g = torch.Generator(device=DEV).manual_seed(5)
    gq, gk = [(1 + 0.1 * torch.randn(D, device=DEV, generator=g)).bfloat16() for _ in range(2)]
    hist = [[[[], []] for _ in range(R)] for _ in range(layers)]  # f64 k, v per layer and request
    ctx = [0] * R
    width = (Hq + 2 * Hkv) * D

    def step(new, run):
        n = sum(new)
        ctx_t, new_t = i32(ctx), i32(new)
        xs = [torch.randn(96, width, device=DEV, generator=g) for _ in range(layers)]
        outs = run(ctx_t, new_t, xs, max(new))
        c.check()
        cu = np.concatenate([[0], np.cumsum(new)])
        for l in range(layers):
            x = xs[l][:n].double().cpu().numpy().reshape(n, Hq + 2 * Hkv, D)
            pos = np.concatenate([ctx[b] + np.arange(new[b]) for b in range(R)])
            turn = lambda y, gamma: norm_rope_ref(y, gamma.double().cpu().numpy(), pos, 1e-5, 5e5)[0]  # noqa: E731
            as16 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).float().bfloat16().double().numpy()  # noqa: E731
            qs = np.stack([as16(turn(x[:, h], gq)) for h in range(Hq)], 1)
            ks = np.stack([as16(turn(x[:, Hq + h], gk)) for h in range(Hkv)], 1)
            vs = as16(x[:, Hq + Hkv:])
            for b in range(R):
                hist[l][b][0][ctx[b]:] = list(ks[cu[b]:cu[b + 1]])
                hist[l][b][1][ctx[b]:] = list(vs[cu[b]:cu[b + 1]])
                for t in range(new[b]):
                    e = ctx[b] + t + 1
                    K, V = np.stack(hist[l][b][0][:e]), np.stack(hist[l][b][1][:e])
                    for h in range(Hq):
                        s = K[:, h // 4] @ qs[cu[b] + t, h] / math.sqrt(D)
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        got = outs[l][cu[b] + t, h].double().cpu().numpy()
                        # a query or key whose f32 value lies within 2^-17 of a rounding border may take the
                        # other bf16 value, a step of 2^-7: about one in 2^9 does, and 2^-12 of a score's
                        # size allows for one in 2^5
                        reach = (np.abs(K[:, h // 4]) @ np.abs(qs[cu[b] + t, h])).max() / math.sqrt(D)
                        size = w @ np.abs(V[:, h // 4])
                        tol = 2.0 ** -8 * size + 2 * (2.0 ** -8 + 2.0 ** -12 * reach) * size
                        assert np.all(np.abs(got - w @ V[:, h // 4]) <= tol)

    def eager(ctx_t, new_t, xs, most):
        c.plan(ctx_t, new_t)
        return [c.attention(l, c.append(l, xs[l], Hq, q_gamma=gq, k_gamma=gk), most) for l in range(layers)]

    def other_stream(ctx_t, new_t, xs, most):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.plan(ctx_t, new_t, stream=s)
        outs = [c.attention(l, c.append(l, xs[l], Hq, q_gamma=gq, k_gamma=gk, stream=s), most, stream=s)
                for l in range(layers)]
        torch.cuda.current_stream().wait_stream(s)
        return outs

    step([20, 33, 1], eager)
    ctx[:] = [20, 33, 1]
    step([1, 1, 1], eager)
    ctx[:] = [21, 34, 2]
    step([4, 2, 3], other_stream)
    ctx[:] = [22, 36, 3]       # two of four, all and one of three drafts stay
    step([0, 1, 3], eager)
    ctx[:] = [0, 37, 6]        # the first request ends; another takes its row
    for l in range(layers):
        hist[l][0] = [[], []]
    step([40, 1, 40], eager)
    ctx[:] = [40, 38, 46]
    held = c.held.tolist()
    assert held == [3, 3, 3] and int(c.free_count) == 24 - 9

    # captured once, replayed with new lengths and inputs
    buf = dict(ctx=i32(ctx), new=i32([1, 1, 1]), xs=[torch.zeros(96, width, device=DEV) for _ in range(layers)])
    graph, outs = torch.cuda.CUDAGraph(), []
    before = (c.table.clone(), c.held.clone(), c.free_count.clone(), c.free_pages.clone())
    with torch.cuda.graph(graph):
        outs = eager(buf["ctx"], buf["new"], buf["xs"], 2)

    def replay(ctx_t, new_t, xs, most):
        buf["ctx"].copy_(ctx_t)
        buf["new"].copy_(new_t)
        for a, b in zip(buf["xs"], xs):
            a.copy_(b)
        graph.replay()
        return outs

    for a, b in zip(before, (c.table, c.held, c.free_count, c.free_pages)):
        assert torch.equal(a, b)
    step([1, 2, 0], replay)
    ctx[:] = [41, 40, 46]
    step([2, 0, 1], replay)


def test_two_calls_on_two_streams_with_their_own_workspaces():
    ctx, new, Hq, Hkv, D, page = [3000, 500], [1, 1], 32, 8, 128, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 21)
    q2 = q.flip(0).contiguous()
    one, two = (paged.attention(x, k, v, table, i32(cu), i32(ctx), 1) for x in (q, q2))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    args = (i32(cu), i32(ctx))
    torch.cuda.synchronize()
    for _ in range(20):
        for i, x in enumerate((q, q2)):
            outs[i].append(paged.attention(x, k, v, table, *args, 1, stream=streams[i]))
    torch.cuda.synchronize()
    for i, want in enumerate((one, two)):
        for o in outs[i]:
            assert torch.equal(o, want)  # the division of the work and the order of joins are fixed


@pytest.mark.parametrize("ctx,new", [([900, 33, 4000], [1, 2, 1]), ([900, 0, 33], [70, 130, 1])])
def test_captured_attention_replays_on_new_inputs_and_repeats_itself(ctx, new):
    """Two graphs of one memory pool, replayed in turn with eager calls between: the same bits as an eager call."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 22)
    args = (i32(cu), i32(ctx), max(new))
    other = (1.5 * torch.randn(q.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))).bfloat16()
    want = [paged.attention(x, k, v, table, *args).clone() for x in (q, other)]
    attention_close(want[1], *attention_ref(other, k, v, table, cu, ctx, page, D ** -0.5), D, is_few(new, Hq, Hkv))
    buf = [torch.zeros_like(q) for _ in range(2)]
    graphs, outs = [], []
    pool = torch.cuda.graph_pool_handle()
    for b in buf:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(paged.attention(b, k, v, table, *args))
        graphs.append(g)
    for first in (0, 1):
        for i in (0, 1):
            buf[i].copy_((q, other)[i ^ first])
        for i in (0, 1):
            graphs[i].replay()
            got = outs[i].clone()
            assert torch.equal(paged.attention(buf[i], k, v, table, *args), got)
            assert torch.equal(got, want[i ^ first])


@pytest.mark.parametrize("new", [[1, 2], [50, 3]])
def test_offsets_past_32_bits_and_a_shared_prefix(new):
    """Pools of 2.6 G elements whose last pages hold the requests; the second request shares the first one's pages
    for its prefix."""
    Hq, Hkv, D, page, pages = 16, 8, 128, 64, 40000
    pool = [torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    assert pool[0].numel() > 1 << 31
    ctx = [300, 130]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    table = torch.full((2, max(need)), -1, dtype=torch.int32, device=DEV)
    table[0, :need[0]] = torch.arange(pages - 1, pages - 1 - need[0], -1, device=DEV)
    table[1, :2] = table[0, :2]                                  # 128 shared tokens
    table[1, 2:need[1]] = torch.arange(pages - 20, pages - 20 - (need[1] - 2), -1, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(9)
    width = (Hq + 2 * Hkv) * D
    # both requests' cached tokens, then the new ones, through the norms and stores
    for lens, at in ((ctx, [0, 128]), (new, ctx)):
        slots, pos = [], []
        for b in range(2):
            first = at[b]
            last = ctx[b] if at[b] != ctx[b] else ctx[b] + new[b]
            for p in range(first, last):
                pos.append(p)
                slots.append(int(table[b, p // page]) * page + p % page)
        x = torch.randn(len(pos), width, device=DEV, generator=g)
        q = paged.qk_norm_rope(x, Hq, Hkv, D, i32(pos), i32(slots), pool[0], pool[1])
    for t in (0, 1):
        p = ctx[0] - 1
        row = pool[t].view(-1)[((int(table[0, p // page]) * Hkv) * page + p % page) * D:][:D]
        assert bool((row != 0).any())
    cu = [0, new[0], sum(new)]
    q = q.clone()
    got = paged.attention(q, pool[0], pool[1], table, i32(cu), i32(ctx), max(new))
    want, size, reach = attention_ref(q, pool[0], pool[1], table, cu, ctx, page, D ** -0.5)
    attention_close(got, want, size, reach, D, is_few(new, Hq, Hkv))


# ------------------------------------------------------------------ refusals of the tensor functions
def test_tensor_functions_refuse_what_does_not_fit():
    q, k, v, table, cu = attention_case([30], [2], 8, 2, 64, 16, 31)
    ok = dict(q=q, kpool=k, vpool=v, table=table, cu=i32(cu), ctx_len=i32([30]), max_new=2)
    paged.attention(**ok)
    for change in (dict(q=q.float()), dict(q=q[:, :7]), dict(q=q.transpose(1, 2)), dict(kpool=k.float()), dict(vpool=v[1:]),
                   dict(kpool=k.transpose(1, 2)), dict(table=table.long()), dict(table=table[0]), dict(cu=i32([0])),
                   dict(ctx_len=torch.zeros(1, dtype=torch.int64, device=DEV)), dict(cu=i32(cu).cpu()),
                   dict(out=torch.empty(3, 8, 64, dtype=torch.bfloat16, device=DEV)),
                   dict(out=torch.empty(2, 8, 64, device=DEV)), dict(status=torch.zeros(1, device=DEV))):
        with pytest.raises((ValueError, L.MkError)):
            paged.attention(**{**ok, **change})
    with pytest.raises(L.MkError) as e:
        paged.attention(**ok, workspace=torch.empty(1024, dtype=torch.uint8, device=DEV))
    assert e.value.code == L.MK_ERR_LIMIT
    x = torch.zeros(2, 12 * 64, device=DEV)
    pos, slots = i32([0, 1]), i32([0, 1])
    for a in ((x.half(), 8, 2, 64, pos, slots, k, v), (x[:, 1:], 8, 2, 64, pos, slots, k, v),
              (x, 8, 2, 64, pos[:1], slots, k, v), (x, 8, 1, 64, pos, slots, k, v), (x, 8, 2, 64, pos.long(), slots, k, v)):
        with pytest.raises((ValueError, L.MkError)):
            paged.qk_norm_rope(*a)
    with pytest.raises(ValueError):
        paged.qk_norm_rope(x, 8, 2, 64, pos, slots, k, v, q_gamma=torch.ones(64, device=DEV))
    with pytest.raises(ValueError):
        paged.plan(pos, pos[:1], table, pos, slots, pos[:1], 16, max_tokens=2)
    with pytest.raises(ValueError):
        paged.plan(pos, pos, i32([[0], [1]]), pos, slots, pos[:1], 16)


def test_empty_calls():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert paged.attention(torch.zeros(0, 8, 64, dtype=torch.bfloat16, device=DEV), k, k, i32([[0]]), i32([0, 0]),
                           i32([5]), 1).shape == (0, 8, 64)
    assert paged.qk_norm_rope(torch.zeros(0, 12 * 64, device=DEV), 8, 2, 64, none, none, k, k).shape == (0, 8, 64)
    out = torch.full((3, 8, 64), 2.0, dtype=torch.bfloat16, device=DEV)
    for most in (1, 50):  # no request has a new token
        paged.attention(out.clone(), k, k, i32([[0], [1]]), i32([0, 0, 0]), i32([5, 0]), most, out=out)
    assert torch.all(out == 2.0)


@pytest.mark.parametrize("bad", [math.nan, -math.inf])
@pytest.mark.parametrize("key", [70, 71, 127, 128, 133, 134, 197, 198, 255, 256, 369])
def test_a_bad_value_reaches_the_rows_that_see_it_and_no_other(key, bad):
    """300 tokens behind 70 keys, four rows to a token: items of 64 tokens, whose first and last keys fall on and
    beside block borders."""
    ctx, new, Hq, Hkv, D, page = [70], [300], 8, 2, 128, 16
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 41)
    want, size, reach = attention_ref(q, k, v, table, cu, ctx, page, D ** -0.5)
    v[int(table[0, key // page]), 1, key % page, 5] = bad
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), 300)
    first = key - ctx[0]  # the first token that sees the key
    seen = got[first:, 4:, 5].float()
    assert bool((torch.isnan(seen) if math.isnan(bad) else seen == bad).all())
    got[first:, 4:, 5] = want[first:, 4:, 5].bfloat16()
    attention_close(got, want, size, reach, D, False)


@pytest.mark.parametrize("G", [1, 3, 4, 7, 8, 16, 48, 128])
def test_attention_with_items_cut_at_every_place(G):
    """Requests of lengths on both sides of the tiles' and blocks' sizes, as many that workers' borders fall anywhere."""
    ctx, new = [0, 1, 127, 128, 255, 900, 0, 383], [9, 130, 128, 1, 33, 2, 257, 64]
    q, k, v, table, cu = attention_case(ctx, new, 2 * G, 2, 64, 32, G)
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new))
    attention_close(got, *attention_ref(q, k, v, table, cu, ctx, 32, 64 ** -0.5), 64, False)


def test_a_tensor_that_requires_a_gradient_is_refused():
    q, k, v, table, cu = attention_case([30], [2], 8, 2, 64, 16, 31)
    args = (k, v, table, i32(cu), i32([30]), 2)
    q.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        paged.attention(q, *args)
    with torch.no_grad():
        paged.attention(q, *args)
    x, pos = torch.zeros(2, 12 * 64, device=DEV), i32([0, 1])
    gain = torch.ones(64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        paged.qk_norm_rope(x, 8, 2, 64, pos, pos, k, v, q_gamma=gain)
    with pytest.raises(ValueError, match="gradient"):
        paged.qk_norm_rope(x.requires_grad_(), 8, 2, 64, pos, pos, k, v)


# ------------------------------------------------------------------ streams, lifetimes, threads
@pytest.mark.parametrize("op", ["plan", "norms", "attention", "verify"])
def test_an_input_dropped_behind_a_call_on_another_stream_is_not_made_over(op):
    """The call's stream is still busy when the input's memory goes back to the allocator and the caller's own stream
    asks for as much again."""
    g = torch.Generator(device=DEV).manual_seed(51)
    if op == "plan":
        source = i32([40, 3, 100])
        new, table, held, free, count = i32([3, 1, 20]), i32([[-1] * 9] * 3), i32([0] * 3), i32(range(20)), i32([20])
        keep = dict(held_out=i32([0] * 3), count_out=i32([0]), max_tokens=30)
        run = lambda x, **kw: paged.plan(x, new, table, held, free, count, 16, **keep, **kw)  # noqa: E731
    elif op == "norms":
        source = torch.randn(40, 12 * 64, device=DEV, generator=g)
        pool = [torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        at = torch.arange(40, dtype=torch.int32, device=DEV)
        run = lambda x, **kw: (paged.qk_norm_rope(x, 8, 2, 64, at, at, *pool, **kw),)  # noqa: E731
    elif op == "attention":
        source, k, v, table, cu = attention_case([300], [3], 8, 2, 64, 16, 51)
        lens = i32(cu), i32([300])
        run = lambda x, **kw: (paged.attention(x, k, v, table, *lens, 3, **kw),)  # noqa: E731
    else:
        from task_graph_interpreter_gb300 import speculative
        source = torch.softmax(torch.randn(3, 4, 1000, device=DEV, generator=g), -1)
        drafts, u = i32([[1, 2, 3]] * 3), torch.full((3, 4), 0.5, device=DEV)
        run = lambda x, **kw: speculative.verify_drafts(x, drafts, u, **kw)  # noqa: E731
    want = [t.clone() for t in run(source.clone())]
    s = torch.cuda.Stream()
    dropped = source.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = run(dropped, stream=s)
    at_address = dropped.data_ptr()
    del dropped
    over = [torch.zeros_like(source) for _ in range(4)]
    assert at_address not in [t.data_ptr() for t in over]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_call_on_a_side_stream_of_a_capture_with_an_input_made_there():
    q, k, v, table, cu = attention_case([300], [3], 8, 2, 64, 16, 53)
    lens = i32(cu), i32([300])
    buf, s, graph = torch.zeros_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = paged.attention(buf * 2, k, v, table, *lens, 3, stream=s)
        over = [torch.zeros_like(q) for _ in range(4)]  # the doubled queries are dropped by now
        torch.cuda.current_stream().wait_stream(s)
    for scale in (0.5, 1.0):
        buf.copy_(q * scale)
        graph.replay()
        assert torch.equal(got, paged.attention(buf * 2, k, v, table, *lens, 3))
    assert not any(bool(t.any()) for t in over)


def test_a_cache_attends_over_the_lengths_it_planned_with():
    """The caller counts its lengths on in place, between the plan and the step's attention."""
    c = paged.PagedCache(1, 8, 16, 2, 64, 2, 4, 64)
    ctx, new = i32([0, 0]), i32([20, 5])
    x = torch.randn(25, 12 * 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(52))
    with pytest.raises(ValueError):  # nothing is planned yet
        c.attention(0, torch.zeros(25, 8, 64, dtype=torch.bfloat16, device=DEV), 20)
    c.plan(ctx, new)
    want = c.attention(0, c.append(0, x, 8), 20).clone()
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        c.plan(ctx, new, stream=stream)
        torch.cuda.synchronize()
        ctx += new
        torch.cuda.synchronize()
        got = c.attention(0, c.append(0, x, 8, stream=stream), 20, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        c.check()
        ctx -= new
    planned = c.ctx_len.clone()
    for wrong in (i32([1, 2, 3]), ctx.long()):  # a refused plan leaves the step before it
        with pytest.raises(ValueError):
            c.plan(wrong, new)
    assert torch.equal(c.ctx_len, planned) and torch.equal(c.attention(0, c.append(0, x, 8), 20), want)


def test_a_cache_is_checked_for_steps_on_every_stream():
    c = paged.PagedCache(1, 4, 16, 2, 64, 1, 4, 2000)
    ctx, new = i32([0]), i32([1000])  # more than its pages hold
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    c.plan(ctx, new, stream=s)
    with pytest.raises(L.MkError) as e:
        c.check()
    assert e.value.code == L.MK_DEV_CAPACITY
    c.check()  # told once
    c.plan(ctx, new, stream=s)  # behind the clearing, whatever the stream
    with pytest.raises(L.MkError):
        c.check()


def test_a_refused_call_in_one_thread_does_not_hold_up_another():
    """The exception's own Python code gives other threads a turn while it is made.  In a process of its own, so that
    a lock held there ends this test and not the run."""
    import os
    import subprocess
    import sys
    code = """
import threading, time
import torch
from task_graph_interpreter_gb300 import _lib as L, paged
q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
args = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[0, 1]], [0, 2], [10])]
raising, refused = threading.Event(), []
plain = L.MkError.__init__
def slow(self, *a):
    raising.set()
    time.sleep(1.0)
    plain(self, *a)
L.MkError.__init__ = slow
def wrong():
    try:
        paged.attention(q, pool, pool, *args, 0)
    except L.MkError as e:
        refused.append(e.code)
t = threading.Thread(target=wrong)
t.start()
assert raising.wait(60)
for most in (2, 3, 4):
    paged.attention(q, pool, pool, *args, most)
torch.cuda.synchronize()
t.join()
assert refused == [L.MK_ERR_ARG], refused
print("both done")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "both done" in r.stdout, r.stderr


def test_a_tensor_that_carries_a_tangent_is_refused():
    """Forward-mode tangents would be lost as silently as gradients, under torch.no_grad() too."""
    import torch.autograd.forward_ad as forward_ad
    from task_graph_interpreter_gb300 import speculative
    q, k, v, table, cu = attention_case([30], [2], 8, 2, 64, 16, 31)
    lens = i32(cu), i32([30])
    x, pos = torch.zeros(2, 12 * 64, device=DEV), i32([0, 1])
    gain = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    p, u, drafts = torch.full((1, 2, 10), 0.1, device=DEV), torch.full((1, 2), 0.5, device=DEV), i32([[3]])
    with forward_ad.dual_level(), torch.no_grad():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: paged.attention(dual(q), k, v, table, *lens, 2),
                     lambda: paged.attention(q, k, dual(v), table, *lens, 2),
                     lambda: paged.qk_norm_rope(dual(x), 8, 2, 64, pos, pos, k, v),
                     lambda: paged.qk_norm_rope(x, 8, 2, 64, pos, pos, k, v, k_gamma=dual(gain)),
                     lambda: speculative.verify_drafts(dual(p), drafts, u),
                     lambda: speculative.verify_drafts(p, drafts, dual(u))):
            with pytest.raises(ValueError, match="tangent"):
                call()
        paged.attention(forward_ad.unpack_dual(dual(q)).primal, k, v, table, *lens, 2)
    with pytest.raises(ValueError, match="gradient"):
        speculative.verify_drafts(p, drafts, u.requires_grad_())


# ------------------------------------------------------------------ long contexts
@pytest.mark.parametrize("heads,n,D,ctx", [(1.0, 9, 128, (1 << 22) - 9), (0.67, 9, 128, (1 << 22) + 77), (1.0, 40, 64, 3 << 20),
                                           (0.67, 9, 64, 1 << 22), (4.0, 1, 128, (1 << 21) - 1), (2.7, 2, 64, 1 << 22)])
def test_attention_over_millions_of_keys_keeps_its_sums(heads, n, D, ctx):
    """As many heads to an SM that a worker sums millions of keys of one item, whole items and cut ones.  The keys are
    1024 distinct ones in turn, from four pages, so the softmax over them is one over 1024 with counts; the values
    have one sign, so that nothing hides what their sums lose.

    Beside the tolerance of shorter contexts: the products cut 2^-22 of the running sum off per 16 keys, twice where
    probabilities are in two parts, over 65536 keys (2^-10 of a sum that grows evenly), and a row's sum of
    probabilities is added up in at most 2^16 steps of 2^-24 (2^-9)."""
    page, Hkv = 256, int(heads * torch.cuda.get_device_properties(0).multi_processor_count)
    g = torch.Generator(device=DEV).manual_seed(n + D)
    k = torch.randn(4, Hkv, page, D, device=DEV, generator=g).bfloat16()
    v = (1 + 0.25 * torch.randn(4, Hkv, page, D, device=DEV, generator=g)).bfloat16()
    q = torch.randn(n, Hkv, D, device=DEV, generator=g).bfloat16()
    table = (torch.arange(-(-(ctx + n) // page), dtype=torch.int32, device=DEV) % 4)[None].contiguous()
    status = i32([0])
    got = paged.attention(q, k, v, table, i32([0, n]), i32([ctx]), n, status=status)
    assert int(status) == 0
    kk, vv = (t.permute(1, 0, 2, 3).reshape(Hkv, 4 * page, D).double() for t in (k, v))
    qq = q.double().transpose(0, 1)                          # [Hkv, n, D]
    seen = ctx + 1 + torch.arange(n, device=DEV)
    count = seen[:, None] // 1024 + (torch.arange(1024, device=DEV)[None] < seen[:, None] % 1024)
    w = torch.softmax(qq @ kk.transpose(1, 2) * D ** -0.5 + count.double().log()[None], -1)
    want, size = (w @ vv).transpose(0, 1), (w @ vv.abs()).transpose(0, 1)
    reach = float((qq.abs() @ kk.abs().transpose(1, 2)).max()) * D ** -0.5
    e = (2.0 ** -16 if n <= 8 else 2.0 ** -8) + reach * (D + 4) * 2.0 ** -23 + 2.0 ** -10 + 2.0 ** -9
    err = (got.double() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + 2 * e * size).all()), f"largest error {float(err.max())}"


@pytest.mark.parametrize("heads,n", [(4.0, 1), (2.7, 8)])
def test_attention_over_millions_of_keys_keeps_its_sums_of_probabilities(heads, n):
    """Two scores in turn, so that every block adds the same amount to a row's sum and is rounded the same way: a lane
    of the few-rows kernel adds eight keys a block, 4 (1 + w), to a sum that reaches 2^19 (1 + w), in steps of 2^-4
    and 2^-3; the heads' weights w put that amount anywhere between two steps.  Within the tolerance of the test
    before, without its allowance for the sum of probabilities."""
    D, page, ctx = 64, 256, (1 << 23) - n
    Hkv = int(heads * torch.cuda.get_device_properties(0).multi_processor_count)
    k = torch.zeros(1, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    # scores 0 and -s (D^-0.5 = 2^-3): weights between 0.2 and 0.9
    s = 8 * torch.linspace(0.1, 1.6, Hkv, device=DEV)
    k[0, :, 1::2, 0] = -s.bfloat16()[:, None]
    v = torch.ones_like(k)
    v[..., 1::2] = -0.7
    q = torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    table = torch.zeros(1, (1 << 23) // page, dtype=torch.int32, device=DEV)
    got = paged.attention(q, k, v, table, i32([0, n]), i32([ctx]), n).double()
    want = v[0, 0, 0].double()  # every value is the same
    tol = (2.0 ** -8 + 2 * (2.0 ** -16 + 2 * 66 * 2.0 ** -23 + 2.0 ** -10)) * want.abs()
    worst = (got - want).abs().amax((0, 1))
    assert bool((worst <= tol).all()), worst.tolist()


MIXED = [  # ctx, new, Hq, Hkv, D: both kernels, cut and whole items, many records and few
    ([4096], [1], 32, 8, 128), ([0, 1000, 0, 64], [700, 33, 0, 256], 32, 4, 64), ([31, 900], [1, 1], 12, 12, 64),
    ([2000], [64], 8, 1, 128), ([513, 100], [4, 2], 4, 2, 128), ([0], [1500], 5, 5, 128), ([5], [2], 32, 1, 64)]


def test_attention_on_a_workspace_of_the_caller():
    """One buffer of the largest size for calls of both kernels in turn, and one of each call's own size, both full of
    NaN and of the call before: the same bits as without."""
    sizes = [paged.attention_workspace(max(new), Hq, Hkv, D).numel() for _, new, Hq, Hkv, D in MIXED]
    shared = torch.full((max(sizes),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for i, (ctx, new, Hq, Hkv, D) in enumerate(MIXED):
            q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, 32, 61 + i)
            args = (q, k, v, table, i32(cu), i32(ctx), max(new))
            status = i32([0])
            want = paged.attention(*args, status=status)
            attention_close(want, *attention_ref(q, k, v, table, cu, ctx, 32, D ** -0.5), D, is_few(new, Hq, Hkv))
            own = torch.full((sizes[i] + 64,), 255, dtype=torch.uint8, device=DEV)
            for ws in (shared, own[:sizes[i]]):
                assert torch.equal(paged.attention(*args, workspace=ws, status=status), want)
            assert torch.all(own[sizes[i]:] == 255) and int(status) == 0
            with pytest.raises(L.MkError) as e:
                paged.attention(*args, workspace=own[:sizes[i] - 1])
            assert e.value.code == L.MK_ERR_LIMIT


def test_calls_that_overlap_on_two_streams_each_with_a_workspace_of_its_own():
    ctx, Hq, Hkv, D, page = [3000, 500], 32, 8, 128, 16
    for new in ([1, 1], [5, 90]):
        q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 71)
        qs = (q, q.flip(0).contiguous())
        lens = i32(cu), i32(ctx)
        wants = [paged.attention(x, k, v, table, *lens, max(new)) for x in qs]
        spaces = [paged.attention_workspace(max(new), Hq, Hkv, D) for _ in range(2)]
        outs = [[torch.zeros_like(q) for _ in range(20)] for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for n in range(20):
            for i in (0, 1):
                paged.attention(qs[i], k, v, table, *lens, max(new), out=outs[i][n], workspace=spaces[i],
                                stream=streams[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(o, wants[i]) for o in outs[i])


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D", [([0, 1000, 0, 64], [700, 33, 0, 256], 32, 4, 64), ([2000], [64], 8, 1, 128),
                                              ([40] * 300, [9] * 300, 4, 1, 128), ([0, 7], [130, 3], 4, 2, 64),
                                              ([4096, 3], [1, 1], 8, 2, 128)])
def test_attention_into_rows_that_are_aligned_to_16_bytes_only(ctx, new, Hq, Hkv, D):
    """Outputs whose rows lie Hq D + 8 elements apart, or that begin 8 elements into the buffer, cut items and whole
    ones: the same bits, and what lies between the rows stays."""
    q, k, v, table, cu = attention_case(ctx, new, Hq, Hkv, D, 16, 81)
    args = (q, k, v, table, i32(cu), i32(ctx), max(new))
    want = paged.attention(*args)
    n, row = cu[-1], Hq * D
    for ld, first in ((row + 8, 0), (row + 16, 8), (row, 8), (row + 24, 8)):
        buf = torch.full((n * ld + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
        out = buf.as_strided((n, Hq, D), (ld, D, 1), first)
        paged.attention(*args, out=out)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert torch.all(buf == 5.0)


def test_a_part_that_takes_longer_than_a_second_is_waited_for():
    """2^28 keys of one head for nine tokens: the kernel's warps for masked values and for the empty second tile wait
    from the part's first block to its last, some 1.5 s.  All keys are the same, so the result is their value."""
    D, page, n = 64, 256, 9
    Hkv, ctx = torch.cuda.get_device_properties(0).multi_processor_count, (1 << 28) - 9
    g = torch.Generator(device=DEV).manual_seed(91)
    k = torch.randn(1, Hkv, 1, D, device=DEV, generator=g).bfloat16().expand(1, Hkv, page, D).contiguous()
    v = torch.randn(1, Hkv, 1, D, device=DEV, generator=g).bfloat16().expand(1, Hkv, page, D).contiguous()
    q = torch.randn(n, Hkv, D, device=DEV, generator=g).bfloat16()
    table = torch.zeros(1, (1 << 28) // page, dtype=torch.int32, device=DEV)
    status = i32([0])
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    got = paged.attention(q, k, v, table, i32([0, n]), i32([ctx]), n, status=status)
    end.record()
    assert int(status) == 0 and start.elapsed_time(end) > 1200.0
    want = v[0, :, 0].double()
    # equal probabilities round alike and cancel; the products' sums lose 2^-11 (see above), the result 2^-8
    assert bool(((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs()).all())


@pytest.mark.parametrize("heads,n,D,lost", [(1.0, 9, 128, 300), (0.67, 40, 64, 600), (4.0, 1, 64, 300), (2.7, 3, 128, 520)])
def test_long_parts_whose_first_pages_are_missing(heads, n, D, lost):
    """Folded results of rows that had seen no key yet count for nothing, whole items and cut ones."""
    page, Hkv, ctx = 256, int(heads * torch.cuda.get_device_properties(0).multi_processor_count), 200000
    g = torch.Generator(device=DEV).manual_seed(lost)
    k, v = (torch.randn(4, Hkv, page, D, device=DEV, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(n, Hkv, D, device=DEV, generator=g).bfloat16()
    pages = torch.arange(-(-(ctx + n) // page), dtype=torch.int32, device=DEV)
    table = torch.where(pages < lost, -1, pages % 4)[None].contiguous()
    status = i32([0])
    got = paged.attention(q, k, v, table, i32([0, n]), i32([ctx]), n, status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    kk, vv = (t.permute(1, 0, 2, 3).reshape(Hkv, 4 * page, D).double() for t in (k, v))
    at = torch.arange(1024, device=DEV)[None]
    upto = lambda m: m // 1024 + (at < m % 1024)  # noqa: E731  (keys among the first m, each page as it comes)
    count = upto((ctx + 1 + torch.arange(n, device=DEV))[:, None]) - upto(torch.tensor([[lost * page]], device=DEV))
    s = q.double().transpose(0, 1) @ kk.transpose(1, 2) * D ** -0.5
    w = torch.softmax(s + count.double().log()[None], -1)
    reach = float((q.double().abs().transpose(0, 1) @ kk.abs().transpose(1, 2)).max()) * D ** -0.5
    want, size = (w @ vv).transpose(0, 1), (w @ vv.abs()).transpose(0, 1)
    # as for shorter contexts, and 2^-10 for what the products' sums lose over 65536 keys
    e = (2.0 ** -16 if n <= 8 else 2.0 ** -8) + reach * (D + 4) * 2.0 ** -23 + 2.0 ** -10
    assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * e * size).all())
