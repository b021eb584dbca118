"""Verification of drafted tokens (mk_verify_drafts of include/mk.h)."""
from __future__ import annotations

from . import _lib as L
from .paged import on_stream


def verify_drafts(p, drafts, u, *, q=None, draft_len=None, tokens=None, accepted=None, status=None, stream=None):
    """Speculative sampling from given random numbers: p f32 [B, K + 1, V] the
    target's probabilities, q f32 [B, K, V] the draft model's (None: drafts
    taken as certain), drafts int32 [B, K] (draft_len[b] of them), u f32
    [B, K + 1].  Returns (tokens int32 [B, K + 1]: the accepted drafts, the
    token drawn behind them, then -1; accepted int32 [B]); given ones may not
    overlap the inputs."""
    args = (p, drafts, u, q, draft_len, tokens, accepted, status)
    return L.calls().verify(*args) if stream is None else on_stream(L.calls().verify, stream, args)
