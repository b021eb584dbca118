"""Verification of drafted tokens against a plain float64 implementation:
whole numbers, equal ones."""
import numpy as np
import pytest
import torch

from task_graph_interpreter_gb300 import _lib as L
from task_graph_interpreter_gb300 import speculative

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ref(p, q, drafts, length, u):
    """numpy: p f32 [B, K+1, V], q f32 [B, K, V] or None -> tokens, accepted; and how far each draw is from a border."""
    B, K = drafts.shape
    V = p.shape[2]
    tokens, accepted, gap = np.full((B, K + 1), -1), np.zeros(B, int), np.ones(B)
    for b in range(B):
        n = K if length is None else min(max(int(length[b]), 0), K)
        t, rejected = 0, False
        while t < n:
            x = int(drafts[b, t])
            if not 0 <= x < V:
                break
            qt = np.float64(q[b, t, x]) if q is not None else 1.0
            if not np.float64(u[b, t]) * qt < np.float64(p[b, t, x]):
                rejected = True
                break
            tokens[b, t] = x
            t += 1
        accepted[b] = t
        row = p[b, t].astype(np.float64)
        less = np.zeros(V)
        if rejected:
            if q is not None:
                less = q[b, t].astype(np.float64)
            else:
                less[drafts[b, t]] = np.inf
        w = np.where(row > less, row - np.where(np.isfinite(less), less, 0.0), 0.0)
        if rejected and not w.sum() > 0:
            w = np.where(row > 0, row, 0.0)
        cum = np.cumsum(w)
        if not cum[-1] > 0:
            continue
        target = np.float64(u[b, K]) * cum[-1]
        hit = np.nonzero((cum > target) & (w > 0))[0]
        tokens[b, t] = hit[0] if len(hit) else np.nonzero(w > 0)[0][-1]
        gap[b] = np.abs(cum - target).min() / cum[-1]
    return tokens, accepted, gap


def case(B, K, V, seed, q=True, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, K + 1, V, generator=g) * sharp
    p = torch.softmax(logits, -1)
    qq = torch.softmax(logits[:, :K] + 0.7 * torch.randn(B, K, V, generator=g), -1) if q else None
    src = qq if q else p[:, :K]
    drafts = torch.multinomial(src.reshape(B * K, V), 1, generator=g).view(B, K).int() if K else torch.zeros(B, 0).int()
    return p, qq, drafts, torch.rand(B, K + 1, generator=g)


def check(p, q, drafts, u, length=None, status=0, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    tokens, accepted = speculative.verify_drafts(kw.get("pd", d(p)), d(drafts), d(u), q=kw.get("qd", d(q)),
                                                 draft_len=d(length), status=st)
    want, acc, gap = ref(p.numpy(), None if q is None else q.numpy(), drafts.numpy(),
                         None if length is None else length.numpy(), u.numpy())
    # the sums are exact to about 2^-45: a draw nearer to a border than that could go either way
    assert gap.min() > 2.0 ** -40
    assert accepted.tolist() == acc.tolist()
    assert tokens.tolist() == want.tolist()
    assert int(st) == status


@pytest.mark.parametrize("B,K,V", [(1, 1, 2), (1, 4, 128256), (3, 8, 1000), (70, 3, 257), (9, 40, 333), (40, 2, 32001),
                                   (2, 5, 4096), (300, 1, 50), (5, 0, 999), (1, 3, 1)])
@pytest.mark.parametrize("with_q", [True, False])
def test_verify_matches_float64(B, K, V, with_q):
    check(*case(B, K, V, B * 100 + K, with_q))


def test_verify_lengths_and_invalid_drafts():
    p, q, drafts, u = case(8, 5, 3001, 3)
    check(p, q, drafts, u, length=torch.tensor([0, 1, 2, 3, 4, 5, 9, -2], dtype=torch.int32))
    u = u * 0.01  # most drafts are accepted: the invalid one is reached
    drafts[2, 3] = -1
    drafts[4, 0] = 3001
    check(p, q, drafts, u, status=L.MK_DEV_BAD_INDEX)


def test_verify_rows_apart_and_unaligned():
    B, K, V = 6, 3, 5003
    p, q, drafts, u = case(B, K, V, 4)
    pd = torch.full((B, K + 1, V + 13), float("nan"), device=DEV)[:, :, 1:V + 1]
    qd = torch.full((B, K, V + 5), float("nan"), device=DEV)[:, :, :V]
    pd.copy_(p)
    qd.copy_(q)
    check(p, q, drafts, u, pd=pd, qd=qd)


def test_verify_draws_at_the_ends():
    """u = 0 takes the first token of any weight, u just under one and beyond the last; a NaN counts as zero."""
    V = 20011
    p = torch.zeros(4, 1, V)
    p[:, 0, 17] = 0.25
    p[:, 0, 9000] = 0.5
    p[:, 0, 19999] = 0.25
    p[:, 0, 20000] = float("nan")
    p[:, 0, 5] = -1.0
    u = torch.tensor([[0.0], [1.0 - 2.0 ** -24], [1.0], [float("nan")]])
    none = torch.zeros(4, 0, dtype=torch.int32)
    tokens, accepted = speculative.verify_drafts(p.to(DEV), none.to(DEV), u.to(DEV))
    assert tokens.flatten().tolist() == [17, 19999, 19999, 17] and accepted.tolist() == [0] * 4


def test_verify_without_anything_to_draw():
    """The target equal to the draft leaves nothing after a rejection: drawn from the target; no weight at all: -1."""
    V = 1500
    p = torch.rand(2, 2, V, generator=torch.Generator().manual_seed(1))
    p[1] = 0.0
    q = p[:, :1].clone()
    u = torch.tensor([[1.0, 0.5], [0.5, 0.5]])  # u q < p fails where p = q and u = 1
    drafts = torch.tensor([[7], [7]], dtype=torch.int32)
    tokens, accepted = speculative.verify_drafts(p.to(DEV), drafts.to(DEV), u.to(DEV), q=q.to(DEV))
    cum = np.cumsum(p[0, 0].double().numpy())
    assert accepted.tolist() == [0, 0]
    assert tokens.tolist() == [[int(np.nonzero(cum > 0.5 * cum[-1])[0][0]), -1], [-1, -1]]


def test_verify_keeps_the_target_distribution():
    """Over many random numbers the first token's frequencies are the target's: 40000 draws of a
    probability w are off by more than 5 sqrt(w (1 - w) / 40000) once in two million."""
    n, V = 40000, 6
    p = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1])
    q = torch.tensor([0.3, 0.05, 0.2, 0.2, 0.05, 0.2])
    g = torch.Generator().manual_seed(9)
    drafts = torch.multinomial(q, n, replacement=True, generator=g).int().view(n, 1)
    u = torch.rand(n, 2, generator=g)
    P = p.expand(n, 2, V).contiguous().to(DEV)
    tokens, _ = speculative.verify_drafts(P, drafts.to(DEV), u.to(DEV), q=q.expand(n, 1, V).contiguous().to(DEV))
    freq = torch.bincount(tokens[:, 0].cpu(), minlength=V).double() / n
    assert torch.all((freq - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / n).sqrt())


def test_verify_captured_and_on_another_stream():
    p, q, drafts, u = (t.to(DEV) for t in case(4, 4, 7000, 5))
    want = speculative.verify_drafts(p, drafts, u, q=q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = speculative.verify_drafts(p, drafts, u, q=q, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = speculative.verify_drafts(p, drafts, u, q=q)
    u.copy_(torch.rand(u.shape, generator=torch.Generator().manual_seed(6)))
    graph.replay()
    want = speculative.verify_drafts(p, drafts, u, q=q)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_verify_without_a_finite_sum_draws_nothing_and_refuses_gradients():
    p = torch.full((2, 1, 5000), 1.0 / 5000, device=DEV)
    p[1, 0, 4000] = float("inf")
    none = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    tokens, accepted = speculative.verify_drafts(p, none, torch.full((2, 1), 0.5, device=DEV))
    assert accepted.tolist() == [0, 0] and 0 <= int(tokens[0, 0]) < 5000 and int(tokens[1, 0]) == -1
    with pytest.raises(ValueError, match="gradient"):
        speculative.verify_drafts(p.requires_grad_(), none, torch.full((2, 1), 0.5, device=DEV))
