"""Verification of drafted tokens (mk_verify_drafts of include/mk.h)."""
from __future__ import annotations

import torch

from . import _lib as L
from .paged import _current_device, _raw_stream, device_of, int32_ptr, on_stream

_F32, _I32 = torch.float32, torch.int32


def _probabilities(t, name, B, rows, V, dev):
    """Elements between the rows of f32 [B, rows, V]."""
    if t.dtype is not _F32 or t.get_device() != dev or t.shape != (B, rows, V):
        raise ValueError(f"{name} must be f32 [{B}, {rows}, {V}] on cuda:{dev}")
    if t.is_contiguous():
        return V
    request, row, one = t.stride()
    if (V > 1 and one != 1) or (B > 1 and rows > 1 and request != rows * row):
        raise ValueError(f"{name} must have evenly spaced contiguous rows")
    return row if rows > 1 else request if B > 1 else V


def verify_drafts(p, drafts, u, *, q=None, draft_len=None, tokens=None, accepted=None, status=None, stream=None):
    """Speculative sampling from given random numbers: p f32 [B, K + 1, V] the
    target's probabilities, q f32 [B, K, V] the draft model's (None: drafts
    taken as certain), drafts int32 [B, K] (draft_len[b] of them), u f32
    [B, K + 1].  Returns (tokens int32 [B, K + 1]: the accepted drafts, the
    token drawn behind them, then -1; accepted int32 [B])."""
    dev = device_of(p, "p")
    if stream is not None or dev != _current_device():
        return on_stream(verify_drafts, dev, stream, (p, drafts, u),
                         dict(q=q, draft_len=draft_len, tokens=tokens, accepted=accepted, status=status))
    if p.dim() != 3 or p.shape[1] < 1:
        raise ValueError("p must be f32 [B, K + 1, V]")
    B, K1, V = p.shape
    K = K1 - 1
    ld_p = _probabilities(p, "p", B, K1, V, dev)
    if K == 0:
        q = None
    ld_q = _probabilities(q, "q", B, K, V, dev) if q is not None else V
    if u.dtype is not _F32 or u.get_device() != dev or u.numel() != B * K1 or not u.is_contiguous():
        raise ValueError(f"u must be contiguous f32 [{B}, {K1}] on cuda:{dev}")
    if drafts.numel() != B * K:
        raise ValueError(f"drafts must be int32 [{B}, {K}]")
    if tokens is None:
        tokens = torch.empty((B, K1), dtype=_I32, device=p.device)
    if accepted is None:
        accepted = torch.empty(B, dtype=_I32, device=p.device)
    if B == 0:
        return tokens, accepted
    L.mk_verify_drafts(_raw_stream(dev), B, K, V, p.data_ptr(), ld_p, 0 if q is None else q.data_ptr(), ld_q,
                       int32_ptr(drafts, "drafts", B * K, dev),
                       0 if draft_len is None else int32_ptr(draft_len, "draft_len", B, dev), u.data_ptr(),
                       int32_ptr(tokens, "tokens", B * K1, dev), int32_ptr(accepted, "accepted", B, dev),
                       0 if status is None else int32_ptr(status, "status", 1, dev))
    return tokens, accepted
