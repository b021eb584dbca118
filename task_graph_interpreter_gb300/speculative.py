"""Verification of drafted tokens (mk_verify_drafts of include/mk.h)."""
from __future__ import annotations

import torch

from . import _lib as L
from .paged import check_device, current_stream, int32_ptr, on_stream, status_ptr


def _probabilities(t, name, B, rows, V, dev):
    """Elements between the rows of f32 [B, rows, V]."""
    if (t.dim() != 3 or t.shape[0] != B or t.shape[1] != rows or t.shape[2] != V or t.dtype is not torch.float32
            or t.device != dev or t.stride(2) != 1 or (B > 1 and t.stride(0) != rows * t.stride(1))):
        raise ValueError(f"{name} must be f32 [{B}, {rows}, {V}] with evenly spaced contiguous rows on {dev}")
    return t.stride(1) if rows > 1 else t.stride(0) if B > 1 else V


def verify_drafts(p, drafts, u, *, q=None, draft_len=None, tokens=None, accepted=None, status=None, stream=None):
    """Speculative sampling from given random numbers: p f32 [B, K + 1, V] the
    target's probabilities, q f32 [B, K, V] the draft model's (None: drafts
    taken as certain), drafts int32 [B, K] (draft_len[b] of them), u f32
    [B, K + 1].  Returns (tokens int32 [B, K + 1]: the accepted drafts, the
    token drawn behind them, then -1; accepted int32 [B])."""
    dev = check_device(p, "p")
    if stream is not None or dev.index != torch.cuda.current_device():
        return on_stream(verify_drafts, dev, stream, p, drafts, u, q=q, draft_len=draft_len, tokens=tokens,
                         accepted=accepted, status=status)
    if p.dim() != 3 or p.shape[1] < 1:
        raise ValueError("p must be f32 [B, K + 1, V]")
    B, K, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    ld_p = _probabilities(p, "p", B, K + 1, V, dev)
    ld_q = _probabilities(q, "q", B, K, V, dev) if q is not None and K else V
    if u.dtype is not torch.float32 or u.numel() != B * (K + 1) or not u.is_contiguous() or u.device != dev:
        raise ValueError(f"u must be contiguous f32 [{B}, {K + 1}] on {dev}")
    if drafts.numel() != B * K:
        raise ValueError(f"drafts must be int32 [{B}, {K}]")
    if tokens is None:
        tokens = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if B == 0:
        return tokens, accepted
    L.mk_verify_drafts(current_stream(dev), B, K, V, p.data_ptr(), ld_p,
                       q.data_ptr() if q is not None and K else 0, ld_q, int32_ptr(drafts, "drafts", B * K, dev),
                       int32_ptr(draft_len, "draft_len", B, dev) if draft_len is not None else 0, u.data_ptr(),
                       int32_ptr(tokens, "tokens", B * (K + 1), dev), int32_ptr(accepted, "accepted", B, dev),
                       status_ptr(status, dev))
    return tokens, accepted
