"""The paged cache in 8 bits against plain float64 implementations: the stores
with a scale for each page and head, attention over e4m3 pages, and a run of
them together.

Tolerances count roundings.  A stored value is off by half a step of e4m3: 2^-4
of it, or 2^-10 of the scale where its code is subnormal; f32 arithmetic before
it as for bf16 pages (2^-17 of the pair's size).  A bf16 result is off by 2^-8 of
its value.  In attention, with A = sum_j w_j |v_j| (w the softmax weights), a
relative error e of every weight moves the result by at most 2 e A (numerator and
sum).  e is 2^-11 for the probabilities' rounding to f16, plus the scores' own
error: queries lose 2^-17 of a row's largest element where the chunk kernel
splits them in two e4m3 parts (times sum |k|), D terms are summed in f32 (2^-23
each, tensor cores truncate) and the exponent is off by 2^-23, both times |score|
sums.  Probabilities under 2^-28 of the largest lose 2^-39 of it in f16.
"""
import math

import numpy as np
import pytest
import torch

from task_graph_interpreter_gb300 import _lib as L
from task_graph_interpreter_gb300 import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def pow2(e):
    """2^e in float64, by its bits (a power function may be a rounding off)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def e4m3(x):
    """float64 rounded to e4m3 values (four significant bits, steps of 2^-9 at least, ties to even)."""
    _, e = torch.frexp(x)
    step = pow2((e - 4).clamp(min=-9))
    return torch.where(torch.isfinite(x), (torch.round(x / step) * step).clamp(-448, 448), x * math.nan)


def pow2_scale(amax):
    m, e = torch.frexp(amax)  # 448 is 0.875 * 2^9
    return pow2(torch.where(amax > 0, (e - 9 + (m > 0.875)).clamp(min=-126), -126))


# ------------------------------------------------------------------ stores
def turned(x, gamma, pos, eps, theta):
    """float64 [N, D]: normed (gamma given) and turned, and the size that f32 errors scale with."""
    D = x.shape[-1]
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    ang = pos.double()[:, None] * theta ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=DEV) / D)
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = x[:, :D // 2], x[:, D // 2:]
    size = a.abs() + b.abs()
    return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([size, size], -1)


def filled(pages, Hkv, page, D, g, spread=1.0, junk=False):
    """A pool with pages of different magnitude, and its scales; `junk`: NaN codes and scales instead."""
    if junk:
        return (torch.full((pages, Hkv, page, D), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3),
                torch.full((pages, Hkv), math.nan, device=DEV))
    x = torch.randn(pages, Hkv, page, D, generator=g, device=DEV) * torch.exp2(
        spread * torch.randn(pages, Hkv, 1, 1, generator=g, device=DEV))
    scale = pow2_scale(x.abs().amax((2, 3)).double()).float()
    return (x / scale[:, :, None, None]).to(E4M3), scale


def check_stores(pool, scale, pool0, scale0, rows, slots, x, size, page):
    """Rows `rows` (in order) of x [N, Hkv, D] float64 were stored at `slots`; everything else stayed."""
    pages, Hkv, _, D = pool.shape
    got, was = pool.double(), pool0.double()
    by_page = {}
    for r in rows:
        by_page.setdefault(slots[r] // page, []).append(r)
    untouched = torch.ones(pages, dtype=torch.bool, device=DEV)
    for pg, mine in by_page.items():
        untouched[pg] = False
        offs = [slots[r] % page for r in mine]
        v, err = x[mine], 2.0 ** -17 * size[mine]  # [n, Hkv, D]
        top, slack = v.abs().amax((0, 2)), err.amax((0, 2))
        lo, hi = pow2_scale((top - slack).clamp(min=0)), pow2_scale(top + slack)
        old = scale0[pg].double()
        if 0 not in offs:
            lo, hi = torch.maximum(lo, old), torch.maximum(hi, old)
        s = scale[pg].double()
        assert bool(((s == lo) | (s == hi)).all()), (pg, s, lo, hi)
        want, tol = v, (2.0 ** -4 * v.abs()).maximum(2.0 ** -10 * s[:, None].expand_as(v)) + err * 1.1
        assert bool(((got[pg][:, offs].transpose(0, 1) * s[:, None] - want).abs() <= tol).all()), pg
        below = [o for o in range(max(offs)) if o not in offs]
        above = [o for o in range(max(offs) + 1, page)]
        held = was[pg][:, below]
        if 0 not in offs:
            again = e4m3(held * (old / s)[:, None, None])
            held = torch.where((s != old)[:, None, None], again, held)
            differ = int((torch.nan_to_num(got[pg][:, below], nan=1e9) != torch.nan_to_num(held, nan=1e9)).sum())
            assert differ == 0, pg
        a, b = pool.view(torch.uint8)[pg][:, above], pool0.view(torch.uint8)[pg][:, above]
        assert torch.equal(a, b)
    assert torch.equal(pool.view(torch.uint8)[untouched], pool0.view(torch.uint8)[untouched])
    assert torch.equal(scale[untouched].view(torch.int32), scale0[untouched].view(torch.int32))


def store_case(ctx, new, Hq, Hkv, D, page, dtype, norm, seed, pad=0, strided=False, gaps=0, junk=False, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    slots, pos = [], []
    need = [-(-(c + n) // page) - c // page if n else 0 for c, n in zip(ctx, new)]
    pages = sum(need) + 3
    ids, at = rng.permutation(pages).tolist(), 0
    for c, n, k in zip(ctx, new, need):
        for t in range(n):
            p = c + t
            slots.append(ids[at + p // page - c // page] * page + p % page)
            pos.append(p)
            if gaps and rng.random() < 0.2:  # rows between a request's that are left out, or not stored
                for _ in range(int(rng.integers(1, gaps + 1))):
                    left = rng.random() < 0.5
                    slots.append(7 if left else -1)
                    pos.append(-1 if left else 5)
        at += k
    slots += [-1] * pad
    pos += [-1] * pad
    N, width = len(slots), (Hq + 2 * Hkv) * D
    qkv = torch.randn(N, width + (24 if strided else 0), device=DEV, generator=g).to(dtype)[:, :width]
    gq, gk = ((1 + 0.1 * torch.randn(D, device=DEV, generator=g)).bfloat16() if w in norm else None for w in "qk")
    kpool, kscale = filled(pages, Hkv, page, D, g, spread, junk)
    vpool, vscale = filled(pages, Hkv, page, D, g, spread, junk)
    return dict(qkv=qkv, pos=pos, slots=slots, gq=gq, gk=gk, kpool=kpool, vpool=vpool, kscale=kscale, vscale=vscale)


def run_store(c, Hq, Hkv, D, page, check=True, eps=1e-5, theta=5e5, status=None):
    qkv, N = c["qkv"], len(c["slots"])
    kp, vp, ks, vs = (c[k].clone() for k in ("kpool", "vpool", "kscale", "vscale"))
    out = torch.full((N, Hq + 1, D), 7.0, dtype=torch.bfloat16, device=DEV)[:, :Hq]
    st = i32([0]) if status is None else status
    paged.qk_norm_rope(qkv, Hq, Hkv, D, i32(c["pos"]), i32(c["slots"]), kp, vp, kscale=ks, vscale=vs, q_gamma=c["gq"],
                       k_gamma=c["gk"], eps=eps, rope_theta=theta, out=out, status=st)
    if check:
        assert int(st) == 0
        x = qkv.double().view(N, Hq + 2 * Hkv, D)
        live = [r for r in range(N) if c["pos"][r] >= 0]
        rows = [r for r in live if c["slots"][r] >= 0]
        pos = torch.tensor(c["pos"], device=DEV).clamp(min=0)
        for h in range(Hq):
            want, size = turned(x[:, h], c["gq"], pos, eps, theta)
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -17 * size + 1e-30
            assert bool(((out[:, h].double() - want).abs() <= tol)[live].all()), h
        dead = [r for r in range(N) if c["pos"][r] < 0]
        assert bool((out[dead] == 7.0).all())
        k = [turned(x[:, Hq + h], c["gk"], pos, eps, theta) for h in range(Hkv)]
        kx, ksize = (torch.stack([a[i] for a in k], 1) for i in (0, 1))
        v = x[:, Hq + Hkv:]
        check_stores(kp, ks, c["kpool"], c["kscale"], rows, c["slots"], kx, ksize, page)
        check_stores(vp, vs, c["vpool"], c["vscale"], rows, c["slots"], v, torch.zeros_like(v), page)
    return out, kp, vp, ks, vs


F32, BF = torch.float32, torch.bfloat16
STORES = [  # ctx, new, Hq, Hkv, D, page, dtype, norm, pad, strided, gaps
    ([0], [1], 32, 8, 128, 64, F32, "qk", 0, False, 0), ([5], [1], 4, 2, 64, 16, F32, "", 3, True, 0),
    ([15, 16, 17, 31, 0], [1] * 5, 12, 12, 64, 16, BF, "k", 0, False, 0),
    ([15, 16, 17, 31, 0, 200], [2, 1, 3, 40, 33, 1], 28, 4, 128, 32, F32, "qk", 23, True, 0),
    ([2 ** 31 - 300], [250], 8, 1, 128, 64, F32, "q", 0, False, 0), ([63, 64, 1], [64, 65, 130], 6, 2, 128, 64, BF, "qk", 5, True, 0),
    ([100, 0], [300, 256], 4, 1, 128, 256, BF, "k", 0, False, 0), ([255, 3], [257, 300], 3, 1, 64, 128, F32, "qk", 1, False, 0),
    ([0], [700], 3, 3, 64, 16, BF, "", 0, False, 0), (list(range(100, 220)), [1] * 120, 8, 2, 128, 16, BF, "qk", 8, False, 0),
    ([17, 30, 0], [40, 100, 64], 4, 2, 128, 64, BF, "qk", 0, False, 3), ([3, 250, 9], [90, 1, 50], 4, 2, 64, 256, F32, "k", 4, True, 15),
    ([0] * 30, list(range(1, 31)), 2, 1, 64, 32, BF, "qk", 0, False, 0),
    ([30, 7, 0], [400, 1, 300], 4, 2, 128, 64, F32, "qk", 9, True, 4), (list(range(600)), [1] * 600, 4, 1, 128, 16, F32, "k", 3, False, 0),
    ([5, 100, 0], [700, 90, 64], 28, 4, 128, 128, BF, "qk", 30, False, 2), ([3] * 200, [1, 5, 2, 9] * 50, 4, 2, 64, 16, BF, "", 0, True, 1),
    ([0, 1], [512, 512], 2, 2, 64, 64, F32, "qk", 0, False, 0), ([77], [3000], 2, 1, 128, 256, BF, "k", 0, False, 0)]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page,dtype,norm,pad,strided,gaps", STORES)
def test_stores_match_float64(ctx, new, Hq, Hkv, D, page, dtype, norm, pad, strided, gaps):
    c = store_case(ctx, new, Hq, Hkv, D, page, dtype, norm, len(ctx) * 31 + page, pad, strided, gaps)
    run_store(c, Hq, Hkv, D, page)


LARGE = [  # as above: keys and values in a launch of their own
    ([0], [700], 16, 8, 128, 64, F32, "qk", 0, False, 0), ([5, 100, 0, 77], [300, 90, 264, 1], 16, 16, 128, 16, BF, "k", 30, True, 0),
    ([30, 7, 0], [400, 1, 300], 32, 32, 64, 32, BF, "", 9, True, 4), (list(range(700)), [1] * 700, 8, 8, 128, 16, F32, "q", 3, False, 0),
    ([255, 3, 64], [257, 300, 130], 16, 16, 64, 128, F32, "qk", 1, False, 2), ([77], [900], 8, 8, 128, 256, F32, "k", 0, False, 15),
    ([3] * 200, [1, 5, 2, 9] * 50, 16, 16, 128, 64, BF, "qk", 0, True, 1)]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page,dtype,norm,pad,strided,gaps", LARGE)
def test_large_stores_match_float64(ctx, new, Hq, Hkv, D, page, dtype, norm, pad, strided, gaps):
    c = store_case(ctx, new, Hq, Hkv, D, page, dtype, norm, len(ctx) * 31 + page, pad, strided, gaps)
    run_store(c, Hq, Hkv, D, page)


def test_a_large_store_holds_what_its_parts_store():
    """The two forms of the launch round alike."""
    c = store_case([0], [1472], 8, 8, 128, 64, BF, "qk", 12, junk=True)
    whole = run_store(c, 8, 8, 128, 64, check=False)
    step = dict(c)
    for a, b in ((0, 640), (640, 1280), (1280, 1472)):
        part = dict(step, qkv=c["qkv"][a:b], pos=c["pos"][a:b], slots=c["slots"][a:b])
        out, *now = run_store(part, 8, 8, 128, 64, check=False)
        # the large form's queries are those of bf16 pages: half a bf16 step of their own
        assert bool(((out.float() - whole[0][a:b].float()).abs() <= 2.0 ** -7 * whole[0][a:b].float().abs() + 2.0 ** -16).all())
        step.update(zip(("kpool", "vpool", "kscale", "vscale"), now))
    for k, w in zip(("kscale", "vscale"), whole[3:]):
        assert torch.equal(step[k].view(torch.int32), w.view(torch.int32))
    for k, w in zip(("kpool", "vpool"), whole[1:3]):
        assert torch.equal(step[k].view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("spread", [0.0, 12.0])
def test_scales_far_below_and_above_the_new_values(spread):
    """Pages begun with scales of 2^-40 to 2^40 times the new values', held codes become subnormal or zero."""
    c = store_case([7, 33, 50, 100, 3], [3, 1, 20, 40, 2], 4, 2, 128, 32, F32, "qk", 5, spread=spread)
    run_store(c, 4, 2, 128, 32)


def test_pages_whose_first_token_is_new_forget_what_they_held():
    c = store_case([0, 32, 64], [5, 32, 70], 4, 2, 128, 32, BF, "qk", 9, junk=True)
    out, kp, vp, ks, vs = run_store(c, 4, 2, 128, 32)
    touched = sorted({s // 32 for s in c["slots"]})
    assert torch.isfinite(ks[touched]).all() and torch.isfinite(vs[touched]).all()


@pytest.mark.parametrize("page,cuts", [(16, [1] * 40), (32, [3, 30, 1, 40, 2]), (64, [64, 1, 1, 62, 20]), (256, [100, 100, 90])])
def test_a_cache_filled_in_steps_holds_what_one_call_stores(page, cuts):
    """Codes and scales do not depend on the steps but where a code became subnormal on the way (off by 2^-9 then)."""
    n, Hq, Hkv, D = sum(cuts), 4, 2, 128
    c = store_case([0], [n], Hq, Hkv, D, page, F32, "qk", 3, junk=True)
    whole = run_store(c, Hq, Hkv, D, page)
    step = dict(c)
    at = 0
    for k in cuts:
        part = dict(step, qkv=c["qkv"][at:at + k], pos=c["pos"][at:at + k], slots=c["slots"][at:at + k])
        out, *now = run_store(part, Hq, Hkv, D, page, check=False)
        assert torch.equal(out, whole[0][at:at + k])
        step.update(zip(("kpool", "vpool", "kscale", "vscale"), now))
        at += k
    last = c["slots"][-1]
    for pool, scale, p1, s1 in ((step["kpool"], step["kscale"], whole[1], whole[3]), (step["vpool"], step["vscale"], whole[2], whole[4])):
        for pg in {s // page for s in c["slots"]}:
            m = last % page + 1 if pg == last // page else page
            assert torch.equal(scale[pg], s1[pg])
            # a code rounded twice: half a subnormal step more
            assert float((pool[pg, :, :m].float() - p1[pg, :, :m].float()).abs().max()) <= 2.0 ** -9


def test_values_that_are_not_finite_are_stored_as_nan():
    c = store_case([0, 20], [20, 30], 4, 2, 64, 32, F32, "", 4)
    c["qkv"][3, (4 + 2) * 64 + 7] = math.inf   # value head 0
    c["qkv"][4, (4 + 3) * 64 + 9] = -math.inf  # value head 1
    c["qkv"][30, (4 + 2) * 64 + 1] = math.nan
    c["qkv"][5, 4 * 64 + 5] = math.inf         # key head 0: its pair turns into inf or NaN
    out, kp, vp, ks, vs = run_store(c, 4, 2, 64, 32, check=False)
    at = lambda pool, r, h: pool.float()[c["slots"][r] // 32, h, c["slots"][r] % 32]  # noqa: E731
    assert torch.isfinite(ks[[s // 32 for s in c["slots"]]]).all() and torch.isfinite(vs[[s // 32 for s in c["slots"]]]).all()
    for r, h, d in ((3, 0, 7), (4, 1, 9), (30, 0, 1)):
        row = at(vp, r, h)
        assert math.isnan(row[d]) and torch.isfinite(torch.cat([row[:d], row[d + 1:]])).all()
    row = at(kp, 5, 0)
    assert torch.isnan(row[[5, 37]]).all() and int(torch.isnan(row).sum()) == 2


def test_zero_and_tiny_and_huge_values():
    c = store_case([0, 0, 0], [4, 4, 4], 1, 1, 64, 16, F32, "", 4)
    c["qkv"][:4] = 0
    c["qkv"][4:8] *= 1e-38
    c["qkv"][8:] *= 1e36
    out, kp, vp, ks, vs = run_store(c, 1, 1, 64, 16)
    assert float(vs[c["slots"][0] // 16, 0]) == 2.0 ** -126 and bool((vp.float()[c["slots"][0] // 16, 0, :4] == 0).all())


def test_rows_that_go_back_in_a_page_and_slots_outside_the_pool_are_reported():
    c = store_case([0], [8], 2, 1, 64, 16, F32, "", 4)
    base = c["slots"][0]
    for slots, stored in (([0, 1, 2, 2, 3, 4, 5, 6], 3), ([4, 5, 3, 4, 6, 7, 8, 9], 2), ([0, 1, 10 ** 6, 2 ** 31 - 1], 2)):
        c2 = dict(c, qkv=c["qkv"][:len(slots)], pos=c["pos"][:len(slots)],
                  slots=[base + s if s < 16 else s for s in slots])
        status = i32([0])
        out, kp, vp, ks, vs = run_store(c2, 2, 1, 64, 16, check=False, status=status)
        assert int(status) == L.MK_DEV_BAD_INDEX
        keep = dict(c2, pos=c2["pos"][:stored], slots=c2["slots"][:stored], qkv=c2["qkv"][:stored])
        out2, kp2, vp2, ks2, vs2 = run_store(keep, 2, 1, 64, 16)
        assert torch.equal(kp.view(torch.uint8), kp2.view(torch.uint8)) and torch.equal(vs, vs2)
        assert torch.equal(vp.view(torch.uint8), vp2.view(torch.uint8)) and torch.equal(ks, ks2)


# ------------------------------------------------------------------ attention
def attention_case(ctx, new, Hq, Hkv, D, page, seed, spread=1.0, spare=3):
    """Codes of requests on scattered pages of different scales; what no request holds is NaN, scales too."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + spare
    ids = torch.randperm(pages, device=DEV, generator=g)
    width = max(need + [1]) + 1
    table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEV)
    pools, scales = [], []
    for _ in range(2):
        pool, scale = filled(pages, Hkv, page, D, g, spread)
        held = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
        at = 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            mine = ids[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine.int()
            held[mine] = torch.arange(need[b] * page, device=DEV).view(-1, page) < c + n
        pool = pool.view(torch.uint8).masked_fill_(~held[:, None, :, None], 0x7F).view(E4M3)
        scale[~held.any(1)] = math.nan
        pools.append(pool)
        scales.append(scale)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (1.5 * torch.randn(cu[-1], Hq, D, device=DEV, generator=g)).bfloat16()
    return q, pools[0], pools[1], scales[0], scales[1], table, cu


def attention_ref(q, kpool, vpool, ks, vs, table, cu, ctx, page, scale, lost=()):
    """float64 (result, sum of weights times |v|, relative error of weights); `lost`: (request, page index) left out."""
    Hq, D = q.shape[1:]
    Hkv = kpool.shape[1]
    G = Hq // Hkv
    out, size = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    reach = lose = top = 0.0
    for b in range(len(ctx)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        Lb = ctx[b] + n
        ids = table[b, : -(-Lb // page)].long().clamp(0, kpool.shape[0] - 1)
        k, v = ((p.view(torch.uint8)[ids].view(E4M3).double() * s[ids].double()[:, :, None, None]).permute(1, 0, 2, 3)
                .reshape(Hkv, -1, D)[:, :Lb] for p, s in ((kpool, ks), (vpool, vs)))
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
            cut = qb[:, h].abs().amax(-1)[:, None] * k[h // G].abs().sum(-1)[None] * scale
            lose = max(lose, float(torch.nan_to_num(cut.masked_fill(~see, 0.0)).max()))
            top = max(top, float(torch.nan_to_num(vv).abs().max()))
    return out, size, 2.0 ** -11 + reach * (D + 4) * 2.0 ** -23 + lose * 2.0 ** -17, top


def close(got, want, size, e, top):
    tol = 2.0 ** -8 * want.abs() + 2 * e * size + 2.0 ** -38 * top + 1e-30
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), f"max excess {float((err - tol).max())}, max error {float(err.max())}"


FEW = [  # ctx, new, Hq, Hkv, D, page
    ([0], [1], 4, 2, 64, 16), ([0], [1], 32, 8, 128, 64), ([1], [1], 8, 1, 128, 16), ([4096], [1], 32, 8, 128, 64),
    ([31, 32, 33, 63, 64, 65], [1] * 6, 32, 8, 128, 32), ([15, 16, 17, 127, 128, 129], [1] * 6, 12, 12, 64, 16),
    ([700, 0, 5, 3000, 12], [1, 0, 1, 1, 0], 28, 4, 128, 16), ([1000, 0, 77], [5, 8, 1], 16, 4, 128, 128),
    ([0, 3, 250], [8, 8, 3], 32, 8, 64, 256), ([333], [1], 32, 1, 64, 32), ([513, 100], [4, 2], 8, 1, 128, 16),
    ([513, 100], [4, 2], 4, 2, 128, 16), ([30, 31, 32, 33], [8, 7, 6, 5], 3, 3, 64, 16), ([100] * 300, [1] * 300, 4, 2, 64, 16),
    ([20000, 9], [1, 1], 40, 8, 128, 16)]
CHUNK = [
    ([0], [9], 4, 1, 64, 16), ([0], [128], 4, 4, 128, 64), ([0], [129], 12, 12, 64, 16), ([5, 0, 300], [40, 1, 77], 32, 8, 128, 32),
    ([0, 1000, 0, 64], [700, 33, 0, 256], 32, 4, 64, 16), ([100, 37], [257, 511], 28, 4, 128, 128),
    ([2000], [64], 8, 1, 128, 256), ([0], [1500], 5, 5, 128, 16), ([127, 128, 129], [127, 128, 129], 6, 2, 64, 64),
    ([50], [30], 96, 1, 64, 32), ([0] * 40, [33 + i for i in range(40)], 8, 2, 128, 16), ([30000], [5], 32, 8, 128, 16)]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", FEW + CHUNK)
def test_attention_matches_float64(ctx, new, Hq, Hkv, D, page):
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, len(ctx) + D)
    status = i32([0])
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), kscale=ks, vscale=vs, status=status)
    assert int(status) == 0
    close(got, *attention_ref(q, k, v, ks, vs, table, cu, ctx, page, D ** -0.5))


@pytest.mark.parametrize("new", [[2, 1, 2], [2, 1, 3], [60, 1, 33]])
def test_attention_strides_and_rows_of_no_request(new):
    """Queries inside a wider row, outputs apart, rows before, between and behind the requests' own; a scale."""
    ctx, Hq, Hkv, D, page = [40, 0, 500], 8, 2, 128, 16
    q0, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 11)
    n = cu[-1]
    wide = torch.full((n + 9, Hq + 4, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[3:3 + n, :Hq] = q0
    out = torch.full((n + 9, Hq + 2, D), 5.0, dtype=torch.bfloat16, device=DEV)
    got = paged.attention(wide[:, :Hq], k, v, table, i32([c + 3 for c in cu]), i32(ctx), max(new), kscale=ks, vscale=vs,
                          out=out[:, :Hq], scale=0.2)
    close(got[3:3 + n], *attention_ref(q0, k, v, ks, vs, table, cu, ctx, page, 0.2))
    assert torch.all(out[:3] == 5.0) and torch.all(out[3 + n:] == 5.0) and torch.all(out[:, Hq:] == 5.0)


@pytest.mark.parametrize("D,page", [(128, 16), (64, 32)])
@pytest.mark.parametrize("new", [[1, 2, 1], [1, 1, 4], [50, 40, 3]])
def test_attention_leaves_out_pages_outside_the_pool(new, D, page):
    ctx, Hq, Hkv = [300, 10, 90], 16, 4
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 12)
    keep = table.clone()
    table[0, 3] = -1
    table[0, 7] = k.shape[0]
    table[1] = 2 ** 31 - 1   # nothing of the second request is there
    status = i32([0])
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), kscale=ks, vscale=vs, status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    lost = [(0, 3), (0, 7)] + [(1, j) for j in range(table.shape[1])]
    close(got, *attention_ref(q, k, v, ks, vs, keep, cu, ctx, page, D ** -0.5, lost))
    assert torch.all(got[cu[1]:cu[2]] == 0)


@pytest.mark.parametrize("new,few", [([1, 1], True), ([40, 20], False)])
@pytest.mark.parametrize("what", ["cu", "past", "max_new", "pages", "negative"])
def test_attention_refuses_lengths_that_do_not_fit(new, few, what):
    ctx, Hq, Hkv, D, page = [30, 40], 8, 2, 64, 16
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 13)
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
    paged.attention(q, k, v, table, i32(cu2), i32(ctx2), most, kscale=ks, vscale=vs, out=out, status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    assert torch.all(out == 5.0)


@pytest.mark.parametrize("shift", [3e4, -3e4])
@pytest.mark.parametrize("new", [[2], [3], [70]])
def test_attention_with_far_apart_scores(new, shift):
    """Scores that jump by thousands from key to key (running maxima move, old sums vanish) and rows of equal scores."""
    ctx, Hq, Hkv, D, page = [400], 4, 1, 128, 16
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, page, 14)
    q.zero_()
    q[:, 0, 0] = 1.0
    q[:, 1, 0] = 64.0
    ids = table[0, : -(-(ctx[0] + new[0]) // page)].long()
    flat = torch.arange(ids.numel() * page, device=DEV, dtype=torch.float32)
    ks[ids, 0] = 2.0 ** 7
    codes = k.view(torch.uint8)
    codes[ids, 0, :, 0] = (flat / flat.numel() * shift / 2 ** 7).view(-1, page).to(E4M3).view(torch.uint8)
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), max(new), kscale=ks, vscale=vs, scale=1.0)
    want, size, _, top = attention_ref(q, k, v, ks, vs, table, cu, ctx, page, 1.0)
    # one product per score, exact in f32; the exponent's error is 2^-23 of the difference to the
    # maximum, which matters only where that is under 150 or so
    close(got, want, size, 2.0 ** -11 + 150 * 2.0 ** -22, top)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("key", [70, 71, 127, 128, 133, 134, 197, 198, 255, 256, 369])
def test_a_nan_reaches_the_rows_that_see_it_and_no_other(key, D):
    for n in (2, 8, 100, 300):
        ctx, Hq, Hkv, page = [370 - n], 4, 1, 16
        q, k, v, ks, vs, table, cu = attention_case(ctx, [n], Hq, Hkv, D, page, 15)
        run = lambda: paged.attention(q, k, v, table, i32(cu), i32(ctx), n, kscale=ks, vscale=vs)  # noqa: E731
        clean = run()
        first = max(0, key - ctx[0])  # the first row that sees the key
        pg = int(table[0, key // page])
        v.view(torch.uint8)[pg, 0, key % page, 5] = 0xFF
        got = run()
        assert torch.equal(got[:first], clean[:first])
        assert torch.isnan(got[first:, :, 5]).all()
        other = [d for d in range(D) if d != 5]
        assert torch.equal(got[first:][..., other], clean[first:][..., other])
        k.view(torch.uint8)[pg, 0, key % page, 3] = 0x7F
        got = run()
        assert torch.equal(got[:first], clean[:first]) and torch.isnan(got[first:]).all()


@pytest.mark.parametrize("n", [2, 60])
def test_queries_of_every_magnitude_and_queries_that_are_not_finite(n):
    ctx, Hq, Hkv, D, page = [200], 4, 1, 128, 32
    q, k, v, ks, vs, table, cu = attention_case(ctx, [n], Hq, Hkv, D, page, 16)
    q[0] *= 2.0 ** 100
    q[1] *= 2.0 ** -120
    ks *= 2.0 ** -104  # scores of the first row are as before, of the others nothing
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), n, kscale=ks, vscale=vs)
    close(got, *attention_ref(q, k, v, ks, vs, table, cu, ctx, page, D ** -0.5))
    q[0, 1, 7] = math.nan
    q[1, 2, 9] = math.inf
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), n, kscale=ks, vscale=vs)
    want, size, e, top = attention_ref(torch.nan_to_num(q, posinf=0.0), k, v, ks, vs, table, cu, ctx, page, D ** -0.5)
    fine = torch.ones(n, Hq, dtype=torch.bool, device=DEV)
    fine[0, 1] = fine[1, 2] = False
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[1, 2]).all()
    close(got[fine], want[fine], size[fine], e, top)


@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_every_magnitude(n, D):
    """Pages whose values' scales are 2^30 apart, zero scales, and scales that are no powers of two."""
    ctx, Hq, Hkv, page = [500], 4, 1, 16
    q, k, v, ks, vs, table, cu = attention_case(ctx, [n], Hq, Hkv, D, page, 17, spread=0.0)
    pages = -(-(500 + n) // page)
    ids = table[0, :pages].long()
    factor = torch.exp2(torch.randint(-15, 16, (pages,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).float())
    vs[ids, 0] *= factor
    ks[ids[3], 0] = 0.0
    vs[ids[4], 0] = 0.0
    args = (q, k, v, table, i32(cu), i32(ctx), n)
    got = paged.attention(*args, kscale=ks, vscale=vs)
    want, size, e, top = attention_ref(q, k, v, ks, vs, table, cu, ctx, page, D ** -0.5)
    # a widened value under 2^-14 loses 2^-25 of the largest scale, of which `top` has at least 1 (its code is 2 or more)
    close(got, want, size + 2.0 ** -13 * top, e, top)
    ks[ids, 0] *= 1.3
    vs[ids, 0] *= 0.77
    got = paged.attention(*args, kscale=ks, vscale=vs)
    want, size, e, top = attention_ref(q, k, v, ks, vs, table, cu, ctx, page, D ** -0.5)
    # the scale's rounding to f16 and the widened value's: 2^-11 each
    close(got, want, size + 2.0 ** -13 * top, e + 2.0 ** -10, top)


@pytest.mark.parametrize("G", [1, 3, 4, 7, 8, 16, 48, 128])
def test_attention_with_items_cut_at_every_place(G):
    ctx, new = [1000 + 37 * i for i in range(23)], [1 + i % 3 for i in range(23)]
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, G, 1, 64, 16, 18)
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), 3, kscale=ks, vscale=vs)
    close(got, *attention_ref(q, k, v, ks, vs, table, cu, ctx, 16, 64 ** -0.5))


@pytest.mark.parametrize("G,n", [(1, 9), (1, 16), (2, 7), (2, 8), (3, 3), (3, 5), (4, 3), (4, 4), (5, 2), (5, 3), (7, 2), (8, 2),
                                 (9, 1), (13, 1), (16, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_of_nine_to_sixteen_rows(G, n, D):
    """Two eights of rows, items cut at every place and whole ones, and one long item whose records two blocks join."""
    for ctx in ([700 + 37 * i for i in range(17)], [20011], [0, 5, 31, 32, 33, 64, 127, 9000]):
        new = [1 + i % n for i in range(len(ctx))][::-1]
        new[0] = n
        q, k, v, ks, vs, table, cu = attention_case(ctx, new, 2 * G, 2, D, 16, G + n)
        got = paged.attention(q, k, v, table, i32(cu), i32(ctx), n, kscale=ks, vscale=vs)
        close(got, *attention_ref(q, k, v, ks, vs, table, cu, ctx, 16, D ** -0.5))


@pytest.mark.parametrize("Hq,n,D,ctx", [(4, 1, 128, (1 << 22) + 5), (4, 2, 64, 3 << 20), (1, 9, 128, (1 << 22) - 9), (1, 40, 64, 3 << 20)])
def test_attention_over_millions_of_keys_keeps_its_sums(Hq, n, D, ctx):
    """Equal scores and values of one: every result is one, whatever the sums have to hold; pages of two scales."""
    page = 256
    pages = -(-(ctx + n) // page)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    k = torch.zeros(pages, 1, page, D, device=DEV).to(E4M3)
    v = torch.full((pages, 1, page, D), 64.0, device=DEV).to(E4M3)
    ks = torch.ones(pages, 1, device=DEV)
    vs = torch.full((pages, 1), 2.0 ** -6, device=DEV)
    v.view(torch.uint8)[1::2] = torch.full((1,), 256.0, device=DEV).to(E4M3).view(torch.uint8)
    vs[1::2] = 2.0 ** -8
    q = torch.ones(n, Hq, D, dtype=torch.bfloat16, device=DEV)
    got = paged.attention(q, k, v, table, i32([0, n]), i32([ctx]), n, kscale=ks, vscale=vs)
    # sums by the products lose 2^-22 per 16 keys at most over the 2^16 that they take alone: 2^-10, and half a bf16 step
    assert float((got.float() - 1).abs().max()) <= 2.0 ** -8


@pytest.mark.parametrize("Hq,n,lost", [(4, 1, 300), (1, 9, 300), (1, 40, 600)])
def test_long_parts_whose_first_pages_are_missing(Hq, n, lost):
    ctx, D, page = 200 * 256 * 6, 128, 256
    pages = -(-(ctx + n) // page)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None].clone()
    table[0, :lost] = -1
    g = torch.Generator(device=DEV).manual_seed(3)
    k, ks = filled(pages, 1, page, D, g, 0.2)
    v, vs = filled(pages, 1, page, D, g, 1.0)
    q = torch.randn(n, Hq, D, device=DEV, generator=g).bfloat16()
    got = paged.attention(q, k, v, table, i32([0, n]), i32([ctx]), n, kscale=ks, vscale=vs)
    keep = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    close(got, *attention_ref(q, k, v, ks, vs, keep, [0, n], [ctx], page, D ** -0.5, [(0, j) for j in range(lost)]))


@pytest.mark.parametrize("new", [[1, 2], [50, 3]])
def test_offsets_past_32_bits_and_a_shared_prefix(new):
    """Pools of more than 2^31 (and 2^32) codes, pages at their far end, and pages that two requests list."""
    Hkv, page, D, ctx = 2, 256, 128, [600, 700]
    pages = (1 << 32) // (Hkv * page * D) + 64
    k = torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    ks, vs = (torch.ones(pages, Hkv, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(1)
    table = torch.full((2, 5), -1, dtype=torch.int32, device=DEV)
    ids = torch.arange(pages - 6, pages, dtype=torch.int32, device=DEV)
    table[0, :3] = ids[:3]
    table[1, :3] = torch.stack([ids[0], ids[3], ids[4]])
    for t, s in ((k, ks), (v, vs)):
        part, sc = filled(6, Hkv, page, D, g)
        t[-6:] = part.view(torch.uint8)
        s[-6:] = sc
    cu = [0, new[0], sum(new)]
    q = torch.randn(cu[-1], 4, D, device=DEV, generator=g).bfloat16()
    got = paged.attention(q, k.view(E4M3), v.view(E4M3), table, i32(cu), i32(ctx), max(new), kscale=ks, vscale=vs)
    near = table.clone()
    near[table >= 0] -= pages - 6
    tail = [t[-6:] for t in (k.view(E4M3), v.view(E4M3), ks, vs)]
    close(got, *attention_ref(q, *tail, near, cu, ctx, page, D ** -0.5))
    # stores at the far end
    qkv = torch.randn(3, 8 * D, device=DEV, generator=g)
    slots = [(pages - 1) * page + 253 + i for i in range(3)]
    k0 = k[-1].clone()
    s0 = ks[-1].clone()
    paged.qk_norm_rope(qkv, 4, Hkv, D, i32([0, 0, 0]), i32(slots), k.view(E4M3), v.view(E4M3), kscale=ks, vscale=vs)
    x = qkv.double().view(3, 8, D)[:, 4:6]
    check_stores(k[-1:].view(E4M3), ks[-1:], k0[None].view(E4M3), s0[None], [0, 1, 2], [253, 254, 255], x,
                 torch.zeros_like(x), page)


def test_captured_calls_replay_on_new_inputs_and_repeat_themselves():
    ctx, new, Hq, Hkv, D, page = [900, 33, 4000], [1, 2, 70], 8, 2, 128, 16
    for most, lens in ((2, [1, 2, 1]), (70, new)):
        q, k, v, ks, vs, table, cu = attention_case(ctx, lens, Hq, Hkv, D, page, 21)
        ws = paged.attention_workspace(most, Hq, Hkv, D, dtype=E4M3)
        cu_t, ctx_t, out = i32(cu), i32(ctx), torch.zeros_like(q)
        call = lambda: paged.attention(q, k, v, table, cu_t, ctx_t, most, kscale=ks, vscale=vs, out=out, workspace=ws)  # noqa: E731,B023
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        q.normal_()
        graph.replay()
        first = out.clone()
        want = attention_ref(q, k, v, ks, vs, table, cu, ctx, page, D ** -0.5)
        close(first, *want)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, first)
        ctx_t.copy_(i32([c - 20 for c in ctx]))
        graph.replay()
        got, eager = out.clone(), call().clone()
        assert torch.equal(got, eager)


# ------------------------------------------------------------------ together
def test_a_serving_loop_over_an_8_bit_cache():
    """Prompts, decodes, drafts rolled back and finished requests through PagedCache, against a cache of the values that
    were stored; then what the step answers: log probabilities from its logits."""
    from task_graph_interpreter_gb300 import logprobs
    Hq, Hkv, D, page, B = 8, 2, 128, 16, 5
    cache = paged.PagedCache(2, 60, page, Hkv, D, B, 24, 400, dtype=E4M3)
    g = torch.Generator(device=DEV).manual_seed(0)
    head = torch.randn(Hq * D, 1000, device=DEV, generator=g) * 0.1
    gk = (1 + 0.1 * torch.randn(D, device=DEV, generator=g)).bfloat16()
    ctx = [0] * B
    hist = [[torch.zeros(0, 2, Hkv, D, device=DEV, dtype=torch.float64) for _ in range(B)] for _ in range(2)]
    steps = [[70, 0, 5, 33, 1], [1, 40, 1, 1, 1], [1, 1, 1, 1, 1], [4, 4, 4, 4, 0], [1, 1, 1, 0, 1], [1, 1, 30, 90, 2]]
    back = {3: [3, 0, 2, 4, 0], 4: [0, 0, 0, 31 + 1 + 1 + 1, 0]}  # tokens rolled back after the step (request 3 ends)
    for t, new in enumerate(steps):
        plan = cache.plan(i32(ctx), i32(new))
        n, cu = sum(new), plan.cu.tolist()
        x = torch.randn(400, (Hq + 2 * Hkv) * D, device=DEV, generator=g) * (1 + t)
        for layer in range(2):
            q = cache.append(layer, x, Hq, k_gamma=gk)
            out = cache.attention(layer, q, max(new))
            for b in range(B):
                pos = torch.arange(ctx[b], ctx[b] + new[b], device=DEV)
                rows = x[cu[b]:cu[b + 1]].double().view(-1, Hq + 2 * Hkv, D)
                k = torch.stack([turned(rows[:, Hq + h], gk, pos, 1e-5, 5e5)[0] for h in range(Hkv)], 1)
                both = torch.stack([k, rows[:, Hq + Hkv:]], 1)
                hist[layer][b] = torch.cat([hist[layer][b][:ctx[b]], both])
                Lb = ctx[b] + new[b]
                if not Lb:
                    continue
                ids = cache.table[b, : -(-Lb // page)].long()
                held = []
                for i, (pool, scale) in enumerate(((cache.kpool, cache.kscale), (cache.vpool, cache.vscale))):
                    s = scale[layer][ids].double()[:, :, None, None]
                    y = (pool[layer].view(torch.uint8)[ids].view(E4M3).double() * s)
                    y = y.permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:Lb]
                    step = (s * torch.ones(1, 1, page, 1, device=DEV)).permute(0, 2, 1, 3).reshape(-1, Hkv, 1)[:Lb]
                    want = hist[layer][b][:Lb, i]
                    # half a step, twice where the scale grew behind a value (its code became subnormal)
                    tol = 2.0 ** -4 * want.abs() + 2.0 ** -9 * step + 2.0 ** -16 * want.abs().amax()
                    assert bool(((y - want).abs() <= tol).all()), (t, layer, b, i)
                    held.append(y.permute(1, 0, 2))
                qb, k, v = q[cu[b]:cu[b + 1]].double(), *held
                see = torch.arange(Lb, device=DEV)[None] <= pos[:, None]
                for h in range(Hq):
                    s = (qb[:, h] @ k[h // 4].T * D ** -0.5).masked_fill(~see, -math.inf)
                    w = torch.softmax(s, -1)
                    want, size = w @ v[h // 4], w @ v[h // 4].abs()
                    got = out[cu[b]:cu[b + 1], h].double()
                    e = 2.0 ** -11 + 2.0 ** -8  # (scores here are under 2^10 in their sums)
                    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2 * e * size + 1e-6).all()), (t, layer, b, h)
        cache.check()
        logits = out[:n].float().view(n, -1) @ head
        tokens = logits.argmax(-1).int()
        r = logprobs.token_logprobs(logits, tokens, top=3)
        want = torch.log_softmax(logits.double(), -1)
        assert torch.equal(r.top_ids[:, 0], tokens)
        assert float((r.logprobs.double() - want.amax(-1)).abs().max()) < 1e-5
        ctx = [c + k - b for c, k, b in zip(ctx, new, back.get(t, [0] * B))]
        if t == 4:
            ctx[3] = 0
    cache.plan(i32([0] * B), i32([0] * B))
    cache.check()
    assert int(cache.free_count) == 60


def test_tensor_functions_refuse_what_does_not_fit():
    q, k, v, ks, vs, table, cu = attention_case([5], [1], 4, 2, 64, 16, 1)
    ok = dict(q=q, kpool=k, vpool=v, table=table, cu=i32(cu), ctx_len=i32([5]), max_new=1, kscale=ks, vscale=vs)
    bf = k.float().bfloat16()
    for change in (dict(kscale=None), dict(vscale=None), dict(kscale=ks[:, :1]), dict(kscale=ks.double()), dict(vscale=vs.cpu()),
                   dict(vscale=vs.t().contiguous().t()), dict(kpool=bf), dict(kpool=bf, vpool=bf), dict(kpool=k[:, :, ::2]),
                   dict(kpool=k.view(torch.uint8), vpool=v.view(torch.uint8)), dict(kscale=3.0),
                   dict(kscale=ks.clone().requires_grad_())):
        with pytest.raises(ValueError):
            paged.attention(**{**ok, **change})
    qkv = torch.zeros(1, 8 * 64, device=DEV)
    ok = dict(qkv=qkv, Hq=4, Hkv=2, D=64, positions=i32([0]), slots=i32([0]), kpool=k, vpool=v, kscale=ks, vscale=vs)
    for change in (dict(kscale=None), dict(vscale=vs[:1]), dict(kpool=bf, vpool=bf), dict(vpool=bf), dict(kscale=ks.half())):
        with pytest.raises(ValueError):
            paged.qk_norm_rope(**{**ok, **change})
    with pytest.raises(ValueError):
        paged.PagedCache(1, 4, 16, 2, 64, 2, 2, 8, dtype=torch.float16)
    with pytest.raises(L.MkError):
        paged.attention(**{**dict(q=q, kpool=k, vpool=v, table=table, cu=i32(cu), ctx_len=i32([5]), max_new=0, kscale=ks,
                                  vscale=vs)})


def test_empty_calls():
    q, k, v, ks, vs, table, cu = attention_case([5], [1], 4, 2, 64, 16, 1)
    none = paged.attention(q[:0], k, v, table, i32([0, 0]), i32([5]), 1, kscale=ks, vscale=vs)
    assert none.shape == (0, 4, 64)
    out = torch.full_like(q, 3.0)
    paged.attention(q, k, v, table, i32([0, 0]), i32([5]), 1, kscale=ks, vscale=vs, out=out)
    assert torch.all(out == 3.0)
    r = paged.qk_norm_rope(torch.zeros(0, 8 * 64, device=DEV), 4, 2, 64, i32([]), i32([]), k, v, kscale=ks, vscale=vs)
    assert r.shape == (0, 4, 64)


def test_calls_on_another_stream_and_two_workspaces():
    a = attention_case([5000, 40], [1, 1], 32, 8, 128, 16, 31)
    b = attention_case([700, 90], [60, 33], 32, 8, 128, 16, 32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    cases = [(a, [5000, 40], 1), (b, [700, 90], 60)]
    dev = [(i32(c[6]), i32(ctx)) for c, ctx, _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got = [paged.attention(c[0], c[1], c[2], c[5], cu, cx, m, kscale=c[3], vscale=c[4], stream=s)
               for (c, _, m), (cu, cx), s in zip(cases, dev, streams)]
    torch.cuda.synchronize()
    for (c, ctx, m), g in zip(cases, got):
        close(g, *attention_ref(c[0], c[1], c[2], c[3], c[4], c[5], c[6], ctx, 16, 128 ** -0.5))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [9, 31, 32, 33])
def test_items_of_one_tile_whose_key_blocks_two_take_in_turn(n, D):
    """One to many blocks of keys, odd and even in number, whole items and cut ones, beside items of two tiles."""
    for ctx in ([0], [100], [128 - n], [129 - n], [256 - n], [257 - n], [300, 0, 600, 1000, 127], [5000, 20], [12345]):
        q, k, v, ks, vs, table, cu = attention_case(ctx, [n] * len(ctx), 8, 2, D, 16, n + ctx[0])
        got = paged.attention(q, k, v, table, i32(cu), i32(ctx), n, kscale=ks, vscale=vs)
        close(got, *attention_ref(q, k, v, ks, vs, table, cu, ctx, 16, D ** -0.5))
    ctx, new = [700, 90, 3000, 0], [n, 80, 5, 200]
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, 8, 2, D, 32, n)
    got = paged.attention(q, k, v, table, i32(cu), i32(ctx), 200, kscale=ks, vscale=vs)
    close(got, *attention_ref(q, k, v, ks, vs, table, cu, ctx, 32, D ** -0.5))


@pytest.mark.parametrize("n,page", [(1, 16), (3, 32), (700, 64)])
def test_a_captured_step_replays_on_new_inputs(n, page):
    """Plan, stores, attention and log probabilities of a step in one graph: the bits of the same step called eagerly,
    with small stores (one launch) and large ones (two, beside each other)."""
    from task_graph_interpreter_gb300 import logprobs
    Hq, Hkv, D, B = 16, 8, 128, 2
    made = [paged.PagedCache(1, 140, page, Hkv, D, B, 64, B * n, dtype=E4M3) for _ in range(2)]
    x = torch.zeros(B * n, (Hq + 2 * Hkv) * D, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(n)
    head = torch.randn(Hq * D, 3000, device=DEV, generator=g) * 0.02
    ctx, new, tokens = i32([0] * B), i32([n] * B), torch.randint(0, 3000, (B * n,), device=DEV, generator=g).int()

    def step(cache):
        cache.plan(ctx, new)
        q = cache.append(0, x, Hq)
        out = cache.attention(0, q, n)
        return q, out, *logprobs.token_logprobs(out.view(B * n, -1).float() @ head, tokens, top=4)

    def start(cache):
        for t in (cache.kpool, cache.vpool):
            t[0].view(torch.uint8).zero_()
        cache.plan(i32([0] * B), i32([0] * B))

    step(made[0])  # (allocations and kernels' first use)
    start(made[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(made[0])
    start(made[1])
    for t in range(3):
        x.normal_(generator=g).mul_(1 + t)
        ctx.fill_(t * n)
        graph.replay()
        want = step(made[1])
        for a, b in zip(got, want):
            assert torch.equal(a, b), t
    for c in made:
        c.check()


# ------------------------------------------------------------------ workspaces, lifetimes, layouts
MIXED = [  # ctx, new, Hq, Hkv, D: both kernels, cut and whole items, many records and few
    ([4096], [1], 32, 8, 128), ([0, 1000, 0, 64], [700, 33, 0, 256], 32, 4, 64), ([31, 900], [1, 1], 12, 12, 64),
    ([8000], [4], 32, 8, 128), ([2000], [64], 8, 1, 128), ([513, 100], [4, 2], 4, 2, 128), ([0], [1500], 5, 5, 128),
    ([5], [2], 32, 1, 64)]


def test_attention_on_a_workspace_of_the_caller():
    """One buffer of the largest size for calls of both kernels in turn, and one of each call's own size, both full of
    NaN and of the call before: the same bits as without."""
    sizes = [paged.attention_workspace(max(new), Hq, Hkv, D, dtype=E4M3).numel() for _, new, Hq, Hkv, D in MIXED]
    shared = torch.full((max(sizes),), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for i, (ctx, new, Hq, Hkv, D) in enumerate(MIXED):
            q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, 32, 61 + i)
            status = i32([0])
            args, kw = (q, k, v, table, i32(cu), i32(ctx), max(new)), dict(kscale=ks, vscale=vs, status=status)
            want = paged.attention(*args, **kw)
            own = torch.full((sizes[i] + 64,), 255, dtype=torch.uint8, device=DEV)
            for ws in (shared, own[:sizes[i]]):
                assert torch.equal(paged.attention(*args, workspace=ws, **kw), want)
            assert torch.all(own[sizes[i]:] == 255) and int(status) == 0
            with pytest.raises(L.MkError) as e:
                paged.attention(*args, workspace=own[:sizes[i] - 1], **kw)
            assert e.value.code == L.MK_ERR_LIMIT


def test_graphs_that_share_a_workspace_replay_one_after_the_other():
    sizes = [paged.attention_workspace(max(new), Hq, Hkv, D, dtype=E4M3).numel() for _, new, Hq, Hkv, D in MIXED]
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device=DEV)
    held = []
    for i, (ctx, new, Hq, Hkv, D) in enumerate(MIXED):
        q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, 64, 91 + i)
        out, lens = torch.zeros_like(q), (i32(cu), i32(ctx))
        call = lambda: paged.attention(q, k, v, table, *lens, max(new), kscale=ks, vscale=vs, out=out, workspace=ws)  # noqa: E731,B023
        want = call().clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        out.zero_()
        held.append((graph, out, want, (q, k, v, ks, vs, table, lens)))
    for order in (range(len(held)), reversed(range(len(held)))):
        for i in order:
            held[i][0].replay()
        for _, out, want, _ in held:
            assert torch.equal(out, want)
            out.zero_()


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D", [([0, 1000, 0, 64], [700, 33, 0, 256], 32, 4, 64), ([2000], [64], 8, 1, 128),
                                              ([40] * 300, [9] * 300, 4, 1, 128), ([0, 7], [130, 3], 4, 2, 64),
                                              ([4096, 3], [1, 1], 8, 2, 128), ([4096, 3], [3, 2], 8, 2, 128)])
def test_attention_into_rows_that_are_aligned_to_16_bytes_only(ctx, new, Hq, Hkv, D):
    q, k, v, ks, vs, table, cu = attention_case(ctx, new, Hq, Hkv, D, 16, 81)
    args, kw = (q, k, v, table, i32(cu), i32(ctx), max(new)), dict(kscale=ks, vscale=vs)
    want = paged.attention(*args, **kw)
    n, row = cu[-1], Hq * D
    for ld, first in ((row + 8, 0), (row + 16, 8), (row, 8), (row + 24, 8)):
        buf = torch.full((n * ld + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
        out = buf.as_strided((n, Hq, D), (ld, D, 1), first)
        paged.attention(*args, out=out, **kw)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert torch.all(buf == 5.0)


@pytest.mark.parametrize("op", ["stores", "attention"])
def test_an_input_dropped_behind_a_call_on_another_stream_is_not_made_over(op):
    if op == "stores":
        g = torch.Generator(device=DEV).manual_seed(51)
        source, at = torch.randn(40, 12 * 64, device=DEV, generator=g), torch.arange(40, dtype=torch.int32, device=DEV)
        pools = [torch.zeros(4, 2, 16, 64, device=DEV).to(E4M3) for _ in range(2)]
        scales = dict(kscale=torch.ones(4, 2, device=DEV), vscale=torch.ones(4, 2, device=DEV))
        run = lambda x, **kw: paged.qk_norm_rope(x, 8, 2, 64, at, at, *pools, **scales, **kw)  # noqa: E731
    else:
        source, k, v, ks, vs, table, cu = attention_case([300], [3], 8, 2, 64, 16, 51)
        lens = i32(cu), i32([300])
        run = lambda x, **kw: paged.attention(x, k, v, table, *lens, 3, kscale=ks, vscale=vs, **kw)  # noqa: E731
    want = run(source.clone()).clone()
    s, dropped = torch.cuda.Stream(), source.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = run(dropped, stream=s)
    at_address = dropped.data_ptr()
    del dropped
    over = [torch.zeros_like(source) for _ in range(4)]
    assert at_address not in [t.data_ptr() for t in over]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_gradient_or_a_tangent_is_refused():
    import torch.autograd.forward_ad as forward_ad
    q, k, v, ks, vs, table, cu = attention_case([30], [2], 8, 2, 64, 16, 31)
    lens, x, pos = (i32(cu), i32([30])), torch.zeros(2, 12 * 64, device=DEV), i32([0, 1])
    attend = lambda a, b, c: paged.attention(a, k, v, table, *lens, 2, kscale=b, vscale=c)  # noqa: E731
    store = lambda a, b, c: paged.qk_norm_rope(a, 8, 2, 64, pos, pos, k, v, kscale=b, vscale=c)  # noqa: E731
    grad = lambda t: t.clone().requires_grad_()  # noqa: E731
    for f, a in ((attend, q), (store, x)):
        for args in ((grad(a), ks, vs), (a, grad(ks), vs), (a, ks, grad(vs))):
            with pytest.raises(ValueError, match="gradient"):
                f(*args)
        with forward_ad.dual_level(), torch.no_grad():
            dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
            for args in ((dual(a), ks, vs), (a, dual(ks), vs), (a, ks, dual(vs))):
                with pytest.raises(ValueError, match="tangent"):
                    f(*args)
        with torch.no_grad():
            f(grad(a), ks, vs)


UNSEEN = [  # ctx, new, Hq, Hkv, D, page: pages begin among the new tokens
    (30, 4, 4, 1, 128, 16), (30, 4, 4, 2, 64, 16), (63, 2, 8, 1, 128, 64), (310, 16, 3, 3, 64, 32), (30014, 4, 8, 2, 128, 16),
    (200, 70, 4, 1, 128, 16), (200, 70, 4, 2, 64, 32), (100, 300, 8, 2, 128, 64), (30014, 6, 4, 1, 128, 16),
    (30014, 6, 4, 1, 64, 32), (0, 500, 12, 12, 64, 16), (127, 128, 6, 2, 128, 128), (250, 20, 16, 1, 128, 256)]


@pytest.mark.parametrize("far", [20, 60])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", UNSEEN)
def test_large_values_of_pages_that_a_row_does_not_see_cost_it_nothing(ctx, new, Hq, Hkv, D, page, far):
    """Values 2^20 and 2^60 times larger from some new token's page on: the rows before it are as exact as without them.
    A key's probability loses 2^-39 (few rows) or 2^-31 (chunks) of the largest, times its value."""
    q, k, v, ks, vs, table, cu = attention_case([ctx], [new], Hq, Hkv, D, page, 21)
    first = min(-(-(ctx + max(1, new // 3)) // page), (ctx + new - 1) // page)  # the first large page
    assert ctx // page < first
    vs[table[0, first:-(-(ctx + new) // page)].long()] *= 2.0 ** far
    got = paged.attention(q, k, v, table, i32(cu), i32([ctx]), new, kscale=ks, vscale=vs)
    want, size, e, _ = attention_ref(q, k, v, ks, vs, table, cu, [ctx], page, D ** -0.5)
    few = new * Hq // Hkv <= 16
    top = 448 * torch.stack([vs[table[0, :(ctx + t) // page + 1].long()].amax(0) for t in range(new)])  # [new, Hkv]
    top = top.double().repeat_interleave(Hq // Hkv, 1)[:, :, None]
    tol = 2.0 ** -8 * want.abs() + 2 * e * size + (2.0 ** -39 if few else 2.0 ** -31) * (ctx + new) * top
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"max excess {float(((err - tol) / top).max())} of the largest value a row sees"


@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_keep_values_far_below_the_largest(D):
    """A row sees keys without weight (scores 400 lower) whose values are 2^60 times those that count."""
    ctx, new, Hq, Hkv, page = 500, 2, 4, 1, 16
    q, k, v, ks, vs, table, cu = attention_case([ctx], [new], Hq, Hkv, D, page, 22)
    ids = table[0, :32].long()
    q.zero_()
    q[:, :, 0] = 1.0
    low = torch.zeros(32, dtype=torch.bool, device=DEV)
    low[[0, 7, 8, 20]] = True
    ks[ids] = 1.0
    k.view(torch.uint8)[ids, 0, :, 0] = torch.where(low, -400.0, 0.0).to(E4M3).view(torch.uint8)[:, None]
    vs[ids[low]] *= 2.0 ** 60
    got = paged.attention(q, k, v, table, i32(cu), i32([ctx]), new, kscale=ks, vscale=vs, scale=1.0)
    assert float(k[ids[low]][..., 0].float().max()) <= -384  # (2^-553 of the others)
    seen = torch.stack([torch.arange(512, device=DEV) <= ctx + t for t in range(new)]).double()
    w = seen * (~low).double().repeat_interleave(page)
    w /= w.sum(-1, keepdim=True)
    val = torch.nan_to_num((v.double() * vs.double()[:, :, None, None])[ids, 0].reshape(512, D)) * (w.sum(0) > 0)[:, None]
    want, size = (w @ val)[:, None], (w @ val.abs())[:, None]
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + D * 2.0 ** -22) * size
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("bits", [22, 26, 30, 36])
@pytest.mark.parametrize("new,D", [(1, 64), (2, 128), (5, 128), (5, 64)])
def test_one_key_above_a_million_others(new, D, bits):
    """A key whose weight is 2^22 to 2^36 times each other's, of which there are 2^20: f16 has few bits left of theirs, or
    none.  Each loses 2^-39 of the largest (few rows) or 2^-31 (chunks) at most."""
    ctx, Hq, Hkv, page = (1 << 20) - new, 4, 1, 64
    pages = (ctx + new) // page
    k = torch.zeros(pages, Hkv, page, D, device=DEV).to(E4M3)
    v = torch.ones(pages, Hkv, page, D, device=DEV).to(E4M3)
    k.view(torch.uint8)[777, 0, 5, 0] = torch.tensor(float(bits), device=DEV).to(E4M3).view(torch.uint8)
    v.view(torch.uint8)[777, 0, 5] = 0
    assert float(k[777, 0, 5, 0].float()) == bits
    ones = torch.ones(pages, Hkv, device=DEV)
    table = torch.randperm(pages, device=DEV).int()[None]
    q = torch.zeros(new, Hq, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1
    scale = 0.98 * math.log(2.0)  # (weights that are no powers of two)
    got = paged.attention(q, k, v, table, i32([0, new]), i32([ctx]), new, kscale=ones, vscale=ones, scale=scale)
    tail = torch.tensor([(ctx + t) * 2.0 ** (-0.98 * bits) for t in range(new)], dtype=torch.float64, device=DEV)
    want = (tail / (1 + tail))[:, None, None]
    e = 2.0 ** -11 + (bits + D + 4) * 2.0 ** -23
    tol = 2.0 ** -8 * want + 2 * e * want + (1 << 20) * 2.0 ** (-39 if new * Hq <= 16 else -31)
    assert bool(((got.double() - want).abs() <= tol).all())


def reordered(c, order):
    index = torch.tensor(order, device=DEV)
    return dict(c, qkv=c["qkv"][index], pos=[c["pos"][r] for r in order], slots=[c["slots"][r] for r in order])


def test_a_slot_outside_the_pool_is_left_out_of_its_page_s_rows():
    """The rows around it are stored as without it: together, at one scale."""
    for ctx, n, Hkv in ((0, 8, 1), (5, 40, 2), (0, 800, 16)):
        c = store_case([ctx], [n], 2 * Hkv, Hkv, 128, 32, F32, "qk", 31)
        for bad in (10 ** 6, 2 ** 31 - 1, c["kpool"].shape[0] * 32):
            order, left = [], set()
            for r in range(n):
                order.append(r)
                if r % 5 == 2:  # a row that goes nowhere behind it
                    left.add(len(order))
                    order.append(r)
            c2 = reordered(c, order)
            c2["slots"] = [bad if i in left else s for i, s in enumerate(c2["slots"])]
            status = i32([0])
            out, *got = run_store(c2, 2 * Hkv, Hkv, 128, 32, check=False, status=status)
            assert int(status) == L.MK_DEV_BAD_INDEX
            _, *want = run_store(c, 2 * Hkv, Hkv, 128, 32)
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


TWO_RUNS = [  # requests' tokens, where the last rows of the first one's page go, heads, page
    ([4, 4], 8, 1, 16), ([9, 30, 30], 69, 2, 16), ([20, 300], 320, 1, 32), ([3, 30, 1100], 500, 16, 64), ([3, 30, 1100], 1133, 16, 16),
    ([100, 100] * 12, 2400, 8, 128)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("new,to,Hkv,page", TWO_RUNS)
def test_a_page_whose_rows_lie_apart_is_reported_and_others_are_stored(new, to, Hkv, page, dtype):
    Hq, D = 2 * Hkv, 64
    c = store_case([0] * len(new), new, Hq, Hkv, D, page, dtype, "qk", 33)
    n = len(c["slots"])
    cut = min(new[0], page) - 2  # the first page's last two rows
    rest = [r for r in range(n) if r not in (cut, cut + 1)]
    at = to - 2
    assert at > cut and c["slots"][rest[at - 1]] // page != c["slots"][0] // page
    apart = reordered(c, rest[:at] + [cut, cut + 1] + rest[at:])
    status = i32([0])
    out, *got = run_store(apart, Hq, Hkv, D, page, check=False, status=status)
    assert int(status) == L.MK_DEV_BAD_INDEX
    # every other page as in the right order; one that the moved rows cut in two may be reported too
    want_out, *want = run_store(c, Hq, Hkv, D, page)
    cut_page = {c["slots"][rest[at - 1]] // page} & {c["slots"][r] // page for r in rest[at:at + 1]}
    others = [pg for pg in range(c["kpool"].shape[0]) if pg != c["slots"][0] // page and pg not in cut_page]
    assert all(torch.equal(a.view(torch.uint8)[others], b.view(torch.uint8)[others]) for a, b in zip(got, want))
    inverse = torch.tensor(rest[:at] + [cut, cut + 1] + rest[at:], device=DEV).argsort()
    assert torch.equal(out[inverse], want_out)


@pytest.mark.parametrize("n,Hkv", [(40, 1), (300, 1), (1500, 8), (5000, 1), (5000, 16), (20000, 1), (40000, 4)])
def test_runs_of_one_row_in_many_pages(n, Hkv):
    """Each row in a page of its own: nothing is reported; then one page comes twice, far apart or behind 16 rows that
    are not stored."""
    D, page = 64, 16
    g = torch.Generator(device=DEV).manual_seed(n)
    slots = torch.randperm(n + 5, device=DEV, generator=g)[:n].int() * page + 3
    qkv = torch.randn(n, 3 * Hkv * D, device=DEV, generator=g).bfloat16()
    pos = torch.full((n,), 3, dtype=torch.int32, device=DEV)
    pools = [torch.zeros(n + 5, Hkv, page, D, device=DEV).to(E4M3) for _ in range(2)]
    scales = [torch.full((n + 5, Hkv), 2.0 ** -20, device=DEV) for _ in range(2)]

    def run(slots, pos):
        status = i32([0])
        paged.qk_norm_rope(qkv, Hkv, Hkv, D, pos, slots, *pools, kscale=scales[0], vscale=scales[1], status=status)
        return int(status)
    assert run(slots, pos) == 0
    v = qkv.view(n, 3, Hkv, D)[:, 2].double()
    want = pow2_scale(v.abs().amax(-1))
    at = slots.long() // page
    assert torch.equal(scales[1][at].double(), want)
    assert torch.equal(pools[1][at][:, :, 3].double(), e4m3(v / want[..., None]))
    for a, b in ((0, n - 1), (n // 2, n // 2 + 2), (n - 3, n - 1)):
        again = slots.clone()
        again[b] = slots[a] + 1
        assert run(again, pos) == L.MK_DEV_BAD_INDEX
    gap = slots.clone()
    gap[-17:] = -1
    gap[-1] = gap[-18] + 1      # behind 16 rows that are not stored
    assert run(gap, pos) == L.MK_DEV_BAD_INDEX
    gap[-2] = gap[-18] + 1      # behind 15: one run
    gap[-1] = -1
    assert run(gap, pos) == 0
    none = pos.clone()
    none[n // 3:n // 3 + 20] = -1  # rows that are left out have no page
    again = slots.clone()
    again[n // 3:n // 3 + 20] = slots[0]
    assert run(again, none) == 0


@pytest.mark.parametrize("pages", [65536, 65537, 200000])
def test_runs_in_pools_of_many_pages(pages):
    n, D, page = 700, 64, 16
    at = torch.linspace(0, pages - 1, n, device=DEV).int()  # the first and the last page among them
    assert torch.unique(at).numel() == n
    pools = [torch.zeros(pages, 1, page, D, device=DEV, dtype=torch.uint8).view(E4M3) for _ in range(2)]
    scales = [torch.full((pages, 1), 2.0 ** -20, device=DEV) for _ in range(2)]
    qkv = torch.randn(n, 3 * D, device=DEV).bfloat16()
    pos = torch.zeros(n, dtype=torch.int32, device=DEV)
    for row, to in ((None, None), (n - 1, 0), (5, n - 1), (300, 400)):
        slots = at * page
        if row is not None:
            slots[row] = slots[to] + 1
        status = i32([0])
        paged.qk_norm_rope(qkv, 1, 1, D, pos, slots, *pools, kscale=scales[0], vscale=scales[1], status=status)
        assert int(status) == (0 if row is None else L.MK_DEV_BAD_INDEX)


@pytest.mark.parametrize("n,Hkv", [(500, 1), (3000, 1), (2000, 16), (20000, 6)])
def test_captured_stores_report_a_page_of_two_runs_on_replay(n, Hkv):
    """Each way of looking for such pages, captured behind what makes its inputs and ahead of what reads its results."""
    D, page = 64, 16
    pages = n // 4 + 2
    c = [torch.zeros(pages, Hkv, page, D, device=DEV, dtype=torch.uint8).view(E4M3) for _ in range(2)]
    scales = [torch.ones(pages, Hkv, device=DEV) for _ in range(2)]
    source, qkv = (torch.randn(n, 3 * Hkv * D, device=DEV).bfloat16() for _ in range(2))
    pos = torch.arange(n, device=DEV).int()
    good = (torch.arange(n, device=DEV) // 4 * page + torch.arange(n, device=DEV) % 4).int()  # four rows a page
    slots, status, out = good.clone(), i32([0]), torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV)
    code, sum_ = i32([0]), torch.zeros(1, device=DEV)

    def step():
        qkv.copy_(source)
        for pool in c:  # (a step with a wrong slot leaves what later ones do not write)
            pool.view(torch.uint8).zero_()
        status.zero_()
        paged.qk_norm_rope(qkv, Hkv, Hkv, D, pos, slots, *c, kscale=scales[0], vscale=scales[1], out=out, status=status)
        code.copy_(status)
        sum_.copy_(c[1].view(torch.uint8).float().sum() + out.float().sum())
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for again in range(3):
        source.normal_()
        slots.copy_(good)
        graph.replay()
        assert int(code) == 0
        want, got = [t.clone() for t in c + scales] + [out.clone()], sum_.clone()
        slots.copy_(good)
        slots[n - 1] = good[4 * again] + 5
        graph.replay()
        assert int(code) == L.MK_DEV_BAD_INDEX
        slots.copy_(good)
        step()
        assert int(code) == 0 and torch.equal(sum_, got)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, c + scales + [out]))


def test_a_scale_that_a_rejected_draft_raised_stays_until_the_page_is_begun_anew():
    c = store_case([3], [3], 2, 1, 64, 16, F32, "", 41)
    c["qkv"][2] *= 2.0 ** 12  # the draft
    after = run_store(c, 2, 1, 64, 16)
    base = c["slots"][0] - 3
    pg = base // 16
    step = dict(c, qkv=c["qkv"][:1] * 0.5, pos=[5], slots=[base + 5], **dict(zip(("kpool", "vpool", "kscale", "vscale"), after[1:])))
    out, kp, vp, ks, vs = run_store(step, 2, 1, 64, 16)  # another token in its place
    assert torch.equal(ks[pg], after[3][pg]) and torch.equal(vs[pg], after[4][pg])
    first = dict(step, pos=[0], slots=[base])            # the page's first token
    out, kp, vp, ks, vs = run_store(first, 2, 1, 64, 16)
    assert bool((ks[pg] * 2 ** 9 <= after[3][pg]).all()) and bool((vs[pg] * 2 ** 9 <= after[4][pg]).all())


@pytest.mark.parametrize("higher", [4, 7, 14])
@pytest.mark.parametrize("new,D", [(1, 64), (2, 128), (3, 64)])
def test_few_rows_keep_small_weights_behind_large_values(new, D, higher):
    """The keys of the first page have no weight, but values 2^4 to 2^14 times the others'; one key has 2^22 times the
    weight of each of the others.  Each weight loses 2^-33 of the largest at most.  So many requests (of the same pages)
    that a worker has a whole one."""
    B, Hq, Hkv, page, pages, bits = 1300, 4, 1, 64, 32, 22
    ctx = pages * page - new
    k = torch.zeros(pages, Hkv, page, D, device=DEV).to(E4M3)
    v = torch.ones(pages, Hkv, page, D, device=DEV).to(E4M3)
    k.view(torch.uint8)[17, 0, 5, 0] = torch.tensor(float(bits), device=DEV).to(E4M3).view(torch.uint8)
    v.view(torch.uint8)[17, 0, 5] = 0
    k.view(torch.uint8)[0, 0, :, 0] = torch.tensor(-448.0, device=DEV).to(E4M3).view(torch.uint8)
    ks, vs = torch.ones(pages, Hkv, device=DEV), torch.ones(pages, Hkv, device=DEV)
    vs[0] = 2.0 ** higher
    table = torch.arange(pages, device=DEV).int().expand(B, pages).contiguous()
    q = torch.zeros(B * new, Hq, D, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1
    cu = (torch.arange(B + 1, device=DEV) * new).int()
    scale = 0.98 * math.log(2.0)
    got = paged.attention(q, k, v, table, cu, i32([ctx] * B), new, kscale=ks, vscale=vs, scale=scale)
    tail = torch.tensor([(ctx + t - page) * 2.0 ** (-0.98 * bits) for t in range(new)], dtype=torch.float64, device=DEV)
    want = (tail / (1 + tail)).repeat(B)[:, None, None]
    e = 2.0 ** -11 + (bits + D + 4) * 2.0 ** -23
    tol = 2.0 ** -8 * want + 2 * e * want + ctx * 2.0 ** -33
    assert bool(((got.double() - want).abs() <= tol).all()), f"{float((got.double() - want).abs().max())}, {float(tol.min())}"
