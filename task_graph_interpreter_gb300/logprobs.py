"""Log probabilities of given tokens (mk_token_logprobs of include/mk.h): what a
server answers with beside the tokens, and how a prompt is scored."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .paged import on_stream


class TokenLogprobs(NamedTuple):
    """Per row: the given token's log probability (None without tokens), the
    entropy in nats, and the ``top`` likeliest tokens [N, top] in descending
    order with their log probabilities."""
    logprobs: Optional[torch.Tensor]
    entropy: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


def token_logprobs(logits, tokens=None, *, top: int = 0, logprobs=None, entropy=None, top_ids=None, top_logprobs=None,
                   status=None, stream=None) -> TokenLogprobs:
    """logits f32 or bf16 [N, V] (rows may lie apart), tokens int32 [N], top at
    most 32.  Of equal logits the lower index comes first.  -inf is no
    probability; a row with a NaN or +inf, or without a finite logit, has NaN
    results.  Rows with a negative token are left out: given results keep what
    they had there (fresh ones hold anything).  A token of V or more gets NaN
    and MK_DEV_BAD_INDEX in ``status``.  Streams, memory and gradients as for
    the operators of ``paged``."""
    args = (logits, tokens, top, logprobs, entropy, top_ids, top_logprobs, status)
    return TokenLogprobs._make(L.calls().logprobs(*args) if stream is None else
                               on_stream(L.calls().logprobs, stream, args))
