"""Token log probabilities against float64.

Tolerance: a logit's difference to the maximum is off by 2^-24 of it in f32, and
its power by that times ln 2 ... in all 2^-22 of the difference and 2^-22 for the
power, so the sum is off by a relative 2^-22 (1 + R), R the range of the logits
that have weight (under 110: smaller powers are zero in f32), plus 2^-24 for each
of the about 30 additions in a row that a term goes through (2^-19); the
logarithm adds 2^-23 of its value.  That is at most 2^-15 in all, and 2^-23 of the
result itself.  The entropy weighs the same errors with differences of up to R
whose weight sums to at most the entropy plus one.
"""
import math

import pytest
import torch

from task_graph_interpreter_gb300 import _lib as L
from task_graph_interpreter_gb300 import logprobs

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 2.0 ** -15


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def check(logits, tokens, top, **given):
    status = i32([0])
    r = logprobs.token_logprobs(logits, tokens, top=top, status=status, **given)
    assert int(status) == 0
    x = logits.double()
    lp = x - torch.logsumexp(x, -1, keepdim=True)
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    ids = torch.sort(logits.float(), dim=-1, descending=True, stable=True).indices[:, :top]
    if tokens is None:
        assert r.logprobs is None
    else:
        want = lp.gather(-1, tokens.long()[:, None])[:, 0]
        near(r.logprobs, want)
    assert bool(((r.entropy.double() - ent).abs() <= TOL * (1 + ent)).all())
    assert torch.equal(r.top_ids.long(), ids)
    near(r.top_logprobs, lp.gather(-1, ids))
    return r


def near(got, want):
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf)
    assert bool(((got.double() - want).abs()[~inf] <= TOL + 2.0 ** -23 * want.abs()[~inf]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,top", [(1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 7, 7), (5, 33, 32), (1, 1000, 5), (7, 1001, 20),
                                     (3, 8191, 1), (2, 8193, 32), (1, 16385, 8), (64, 32000, 5), (1, 128256, 32),
                                     (150, 128256, 20), (40, 50257, 3), (700, 5003, 2), (2, 1000003, 32)])
def test_matches_float64(N, V, top, dtype):
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn(N, V, device=DEV, generator=g) * 3).to(dtype)
    tokens = torch.randint(0, V, (N,), device=DEV, generator=g).int()
    check(x, tokens, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_rows_at_every_alignment_and_apart(offset, dtype):
    g = torch.Generator(device=DEV).manual_seed(offset)
    wide = torch.full((9, 9011), math.nan, dtype=dtype, device=DEV)
    x = wide[:, offset:offset + 8999]
    x.copy_(torch.randn(9, 8999, device=DEV, generator=g) * 2)
    tokens = i32([0, 8998, 1, 7, 8, 8990, 3, 4, 5])
    check(x, tokens, 9)
    x[:, 0] = 20    # the row's ends are the likeliest
    x[:, -1] = 21
    check(x, tokens, 9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["up", "down", "equal", "steps", "saw", "zeros"])
@pytest.mark.parametrize("V", [300, 8200, 70000])
def test_orders_that_flood_the_candidates(kind, V, dtype):
    """Ascending logits (each step's are larger than all before), equal ones (ties go to the lowest index), and zeros of
    both signs (equal)."""
    i = torch.arange(V, device=DEV, dtype=torch.float32)
    row = {"up": i / V * 50, "down": -i / V * 50, "equal": torch.zeros_like(i), "steps": torch.floor(i / 100) / V * 5000,
           "saw": (i * 7919 % V) / V * 40, "zeros": torch.where(i % 3 == 0, 0.0, -0.0)}[kind]
    x = row.to(dtype).expand(4, V).clone()
    check(x, i32([0, V - 1, V // 2, 5]), 32)


@pytest.mark.parametrize("V", [50, 20000, 128256])
def test_masked_vocabularies(V):
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.full((6, V), -math.inf, device=DEV)
    few = [1, 2, 5, 40, 3, V // 2]
    tokens = []
    for r, n in enumerate(few):
        ids = torch.randperm(V, device=DEV, generator=g)[:n]
        x[r, ids] = torch.randn(n, device=DEV, generator=g) * 4
        tokens.append(int(ids[0]))
    r = check(x, i32(tokens), 20)
    assert float(r.entropy[0]) == 0.0 and float(r.logprobs[0]) == 0.0
    check(x.bfloat16(), i32(tokens), 20)
    # a token that is masked
    other = i32([(t + 1) % V for t in tokens])
    got = logprobs.token_logprobs(x[:1], other[:1]).logprobs
    assert float(got) == -math.inf


@pytest.mark.parametrize("V", [40, 9000, 128256])
def test_rows_that_are_not_finite(V):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(5, V, device=DEV, generator=g)
    x[1, V // 2] = math.nan
    x[2, V - 1] = math.inf
    x[3] = -math.inf
    x[4] = math.nan
    r = logprobs.token_logprobs(x, i32([1] * 5), top=3)
    assert torch.isfinite(r.logprobs[0]) and torch.isnan(r.logprobs[1:]).all()
    assert torch.isfinite(r.entropy[0]) and torch.isnan(r.entropy[1:]).all()
    assert torch.isnan(r.top_logprobs[1:]).all()
    clean = torch.where(torch.isnan(x[1]), -math.inf, x[1])
    assert r.top_ids[1].tolist() == torch.topk(clean, 3).indices.tolist()
    assert int(r.top_ids[2, 0]) == V - 1 and r.top_ids[3].tolist() == [0, 1, 2] and r.top_ids[4].tolist() == [-1] * 3


def test_large_logits_and_far_apart_ones():
    g = torch.Generator(device=DEV).manual_seed(4)
    for scale, shift in ((1e-20, 0), (1.0, 1000.0), (1.0, -30000.0), (1e4, 0), (1e30, 0)):
        x = torch.randn(3, 12345, device=DEV, generator=g) * scale + shift
        check(x, x.argmax(-1).int(), 8)


def test_rows_without_a_token_are_left_out():
    x = torch.randn(6, 1000, device=DEV)
    given = dict(logprobs=torch.full((6,), 7.0, device=DEV), entropy=torch.full((6,), 7.0, device=DEV),
                 top_ids=torch.full((6, 4), 7, dtype=torch.int32, device=DEV), top_logprobs=torch.full((6, 4), 7.0, device=DEV))
    status = i32([0])
    r = logprobs.token_logprobs(x, i32([3, -1, 5, -7, 999, 1000]), top=4, status=status, **given)
    assert int(status) == L.MK_DEV_BAD_INDEX
    for k, v in given.items():
        assert getattr(r, k).data_ptr() == v.data_ptr()
        assert torch.all(v[[1, 3]] == 7) and not torch.any(v[[0, 2, 4]] == 7.0)
    assert torch.isnan(r.logprobs[5]) and torch.isfinite(r.entropy[5]) and torch.isfinite(r.top_logprobs[5]).all()


def test_without_tokens_and_without_alternatives():
    x = torch.randn(5, 3001, device=DEV)
    check(x, None, 6)
    r = check(x, None, 0)
    assert r.top_ids.shape == (5, 0)
    assert logprobs.token_logprobs(x[:0], i32([]), top=3).top_ids.shape == (0, 3)


def test_results_do_not_depend_on_the_split_of_a_row():
    """The same row alone (in parts on eight CTAs) and among many (on one): the same alternatives, sums to rounding."""
    x = torch.randn(2000, 20011, device=DEV)
    x[:, 100:200] = 3.0
    many = logprobs.token_logprobs(x, i32([5] * 2000), top=32)
    for r in (0, 1, 1999):
        one = logprobs.token_logprobs(x[r:r + 1], i32([5]), top=32)
        assert torch.equal(one.top_ids[0], many.top_ids[r])
        assert float((one.logprobs[0] - many.logprobs[r]).abs()) <= 2 * TOL
    again = logprobs.token_logprobs(x, i32([5] * 2000), top=32)
    assert all(torch.equal(a, b) for a, b in zip(many, again))


def test_captured_and_on_another_stream():
    x = torch.randn(33, 128256, device=DEV)
    tokens = torch.randint(0, 128256, (33,), device=DEV).int()
    out = logprobs.token_logprobs(x, tokens, top=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logprobs.token_logprobs(x, tokens, top=5, **out._asdict())
    x.normal_()
    graph.replay()
    fresh = logprobs.token_logprobs(x, tokens, top=5)
    assert all(torch.equal(a, b) for a, b in zip(out, fresh))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = logprobs.token_logprobs(x, tokens, top=5, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, fresh))


def test_tensor_functions_refuse_what_does_not_fit():
    x, t = torch.randn(4, 100, device=DEV), i32([0] * 4)
    f = logprobs.token_logprobs
    for args, kw in (((x.cpu(), t), {}), ((x.half(), t), {}), ((x[0], t), {}), ((x.t(), t), {}), ((x, t[:3]), {}),
                     ((x, t.long()), {}), ((x, t), dict(top=33)), ((x, t), dict(top=-1)), ((x[:, :3], t), dict(top=4)),
                     ((x[:, :0], t), {}), ((x, t), dict(entropy=torch.zeros(3, device=DEV))),
                     ((x, t), dict(top=2, top_ids=torch.zeros(4, 2, device=DEV))),
                     ((x, t), dict(top=2, top_logprobs=torch.zeros(2, 4, device=DEV).t())),
                     ((x, None), dict(logprobs=torch.zeros(4, device=DEV))), ((x.clone().requires_grad_(), t), {})):
        with pytest.raises(ValueError):
            f(*args, **kw)
    with pytest.raises(L.MkError):  # rows that overlap
        f(x[:1].expand(4, 100), t)


def test_a_tensor_that_carries_a_tangent_is_refused():
    import torch.autograd.forward_ad as forward_ad
    x, t = torch.randn(4, 100, device=DEV), i32([0] * 4)
    with forward_ad.dual_level(), torch.no_grad():
        with pytest.raises(ValueError, match="tangent"):
            logprobs.token_logprobs(forward_ad.make_dual(x, torch.ones_like(x)), t)
    with torch.no_grad():
        logprobs.token_logprobs(x.requires_grad_(), t)


def test_logits_dropped_behind_a_call_on_another_stream_are_not_made_over():
    x = torch.randn(20, 30011, device=DEV)
    t = torch.randint(0, 30011, (20,), device=DEV).int()
    want = logprobs.token_logprobs(x, t, top=7)
    s, dropped = torch.cuda.Stream(), x.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = logprobs.token_logprobs(dropped, t, top=7, stream=s)
    at = dropped.data_ptr()
    del dropped
    over = [torch.zeros_like(x) for _ in range(4)]
    assert at not in [o.data_ptr() for o in over]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_that_overlap_on_two_streams():
    xs = [torch.randn(n, 128256, device=DEV) for n in (1, 30)]
    ts = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (1, 30)]
    want = [logprobs.token_logprobs(x, t, top=20) for x, t in zip(xs, ts)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[logprobs.token_logprobs(x, t, top=20, stream=s) for x, t, s in zip(xs, ts, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for both in got:
        for a, b in zip(both, want):
            assert all(torch.equal(c, d) for c, d in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_offsets_past_32_bits(dtype):
    """Rows 2^29 and more elements apart: the last begins behind 2^32 bytes."""
    ld, N, V = (1 << 29) + 7, 4 if dtype == torch.float32 else 8, 1003
    x = torch.zeros((N - 1) * ld + V, dtype=dtype, device=DEV).as_strided((N, V), (ld, 1))
    x.copy_(torch.randn(N, V, device=DEV))
    assert (N - 1) * ld * x.element_size() > 1 << 32
    check(x, i32([3] * N), 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [0.0, -1e38, -1e34, -3e30])  # 0: the type's lowest value
@pytest.mark.parametrize("N,V", [(3, 300), (3, 20011), (3, 128256), (200, 9001)])
def test_vocabularies_masked_with_finite_values(N, V, low, dtype):
    """Masks of the type's lowest value, and of others so low that their number times their distance to an ordinary
    logit is past the largest f32: without weight, whether threads, warps or parts hold nothing else."""
    g = torch.Generator(device=DEV).manual_seed(V)
    low = low or torch.finfo(dtype).min
    x = torch.full((N, V), low, device=DEV).to(dtype)
    x[0, -5:] = torch.tensor([3, 1, -2, 5, 0.5], device=DEV).to(dtype)  # ordinary ones last
    some = torch.randperm(V, device=DEV, generator=g)[:V // 50 + 1]     # scattered
    x[1:, some] = (4 * torch.randn(N - 1, some.numel(), device=DEV, generator=g)).to(dtype)
    tokens = torch.full((N,), V - 4, dtype=torch.int32, device=DEV)
    tokens[1:] = some[0].int()
    check(x, tokens, 5)
    x[0, 7] = 1e38  # an ordinary one is as far from the largest
    x[-1] = x[-1].flip(0)
    r = logprobs.token_logprobs(x, None, top=1)
    assert int(r.top_ids[0, 0]) == 7 and float(r.entropy[0]) == 0.0 and float(r.top_logprobs[0, 0]) == 0.0
    assert bool(torch.isfinite(r.entropy).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [300, 128256])
def test_rows_of_lowest_values_alone_are_uniform(V, dtype):
    low = torch.finfo(dtype).min
    x = torch.full((2, V), low, device=DEV).to(dtype)
    x[1, V // 3:] = -math.inf
    r = logprobs.token_logprobs(x, i32([V // 4, V // 4]), top=3)
    want = torch.tensor([math.log(V), math.log(V // 3)], dtype=torch.float64, device=DEV)
    near(r.logprobs, -want)
    assert bool(((r.entropy.double() - want).abs() <= TOL * (1 + want)).all())
    near(r.top_logprobs, -want[:, None].expand(2, 3))
    assert r.top_ids.tolist() == [[0, 1, 2]] * 2
