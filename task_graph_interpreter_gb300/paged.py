"""A paged KV cache: block tables and slot maps, per-head norms with rotation
and page stores, and attention of new tokens over the pages (the operators
mk_paged_plan, mk_qk_norm_rope and mk_paged_attention of include/mk.h).

The functions take PyTorch tensors on one CUDA device (not necessarily the
current one) and enqueue on that device's current stream, or on ``stream``;
nothing synchronises.  With ``stream`` they behave as under
``torch.cuda.stream(stream)``: the caller orders that stream behind whatever
made the inputs, and other streams behind it before they use the results; fresh
results are its memory.  Tensors that the caller passes may be dropped as soon
as the call returns: their memory is not given out again before ``stream`` is
through with them.  Tensors that do not fit raise ValueError, what the library
refuses MkError (the checks are in csrc_ops/calls.cpp).

Lengths, tables and maps are int32 tensors that the GPU reads; what is wrong
with their values is reported in ``status`` (an int32 device tensor, zeroed by
the caller, that receives the first MK_DEV_* code) and nowhere else: without
one, rows that a wrong length left unwritten look like any others.  The
operators serve inference: a tensor that requires a gradient is refused outside
``torch.no_grad()``, one that carries a forward-mode tangent altogether.
``PagedCache`` holds a cache's pools, tables and free pages and runs the
operators on them.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib as L


def on_stream(fn, stream, args):
    """Call ``fn`` with ``stream`` current; the tensors have to be on its device.  The allocator learns that
    ``stream`` uses them: their memory may belong to another stream, which would hand it out again while the call
    still waits."""
    tensors = [t for t in args if isinstance(t, torch.Tensor) and t.is_cuda]
    if any(t.device != stream.device for t in tensors):
        raise ValueError(f"the stream is on {stream.device}, a tensor is not")
    for t in tensors:
        t.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(*args)


class Plan(NamedTuple):
    """What a step's new tokens are: ``cu`` [B + 1] exclusive sums of their
    counts, their ``positions`` and ``slots`` [max_tokens] (-1 behind the
    last)."""
    cu: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor


def plan(ctx_len, new_len, table, held, free_pages, free_count, page_size: int, *, cu=None, positions=None, slots=None,
         max_tokens: int = None, held_out=None, count_out=None, status=None, stream=None) -> Plan:
    """Block tables and slot maps of a step (mk_paged_plan): request b has
    ctx_len[b] cached and new_len[b] new tokens and holds held[b] pages,
    listed in table[b]; pages it no longer needs go back on the stack
    free_pages[:free_count], then missing ones come from its top.  ``held``
    and ``free_count`` are updated in place unless ``held_out`` and
    ``count_out`` are given.  A page has one holder: one that two requests
    hold would go back on the stack twice.  ``positions`` and ``slots`` (or
    ``max_tokens``) set how many new tokens the step can have."""
    args = (ctx_len, new_len, table, held, held_out, free_pages, free_count, count_out, page_size, cu, positions,
            slots, max_tokens, status)
    return Plan._make(L.calls().plan(*args) if stream is None else on_stream(L.calls().plan, stream, args))


def qk_norm_rope(qkv, Hq: int, Hkv: int, D: int, positions, slots, kpool, vpool, *, q_gamma=None, k_gamma=None,
                 eps: float = 1e-5, rope_theta: float = 5e5, out=None, status=None, stream=None):
    """RMS norms of queries and keys for each head (none where its gain is
    None), the rotate-half rotary embedding at ``positions``, and the stores
    of keys and values at ``slots`` (mk_qk_norm_rope).  qkv f32 or bf16
    [N, (Hq + 2 Hkv) D], rows may lie apart; returns the queries, bf16
    [N, Hq, D] (``out`` if given, which may not overlap qkv).  Rows with a
    negative position are left out; ``out`` keeps what it had there (a fresh
    one holds anything)."""
    args = (qkv, Hq, Hkv, D, positions, slots, kpool, vpool, q_gamma, k_gamma, eps, rope_theta, out, status)
    return L.calls().qk_norm_rope(*args) if stream is None else on_stream(L.calls().qk_norm_rope, stream, args)


def attention_workspace(max_new: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    """A workspace for ``attention`` with these sizes.  Calls that share one
    must not overlap: run them on one stream."""
    with torch.cuda.device(device):
        return torch.empty(L.mk_paged_attention_workspace(max_new, Hq, Hkv, D), dtype=torch.uint8, device=device)


def attention(q, kpool, vpool, table, cu, ctx_len, max_new: int, *, scale: float = None, out=None, workspace=None,
              status=None, stream=None):
    """Attention of the requests' new tokens over their pages, causal among
    the new ones (mk_paged_attention).  q bf16 [N, Hq, D] (rows may lie
    apart), row cu[b] + t is token t of request b, which sees the keys at
    positions 0 .. ctx_len[b] + t of the pages table[b]; no request has more
    than ``max_new`` new tokens.  Returns ``out`` bf16 [N, Hq, D]; rows of no
    request keep what it had (a fresh one holds anything).  Without a
    ``workspace`` one is taken from PyTorch's allocator for the call.
    ``out`` may not overlap q.

    With max_new Hq / Hkv <= 8 probabilities keep 2^-16, beyond it they are
    rounded to bf16 (results off by 1.7e-3 and 2.1e-3 to 2.4e-3, their own
    rounding included).  That goes for the whole call: a single token beside
    a prompt is computed as the prompt is, unless it has a call of its own."""
    args = (q, kpool, vpool, table, cu, ctx_len, max_new, scale, out, workspace, status)
    return L.calls().attention(*args) if stream is None else on_stream(L.calls().attention, stream, args)


class PagedCache:
    """The KV cache of ``layers`` layers in pages, for up to ``max_requests``
    requests and ``max_tokens`` new tokens a step.  Per step: ``plan`` with
    the requests' lengths, then per layer ``append`` (norms, rotation, page
    stores) and ``attention``.  A request that ends, or whose drafts were
    rejected, gives its pages back through the next plan's lengths.  No two
    requests may hold the same page.  ``check`` tells of lengths that did not
    fit.  The cache is made on the current stream, and its steps follow one
    another: the caller orders a step on another stream behind both."""

    def __init__(self, layers: int, num_pages: int, page_size: int, Hkv: int, D: int, max_requests: int,
                 max_pages: int, max_tokens: int, device="cuda"):
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.page_size, self.Hkv, self.D = page_size, Hkv, D
        shape = (num_pages, Hkv, page_size, D)
        self.kpool = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(layers)]
        self.vpool = [torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(layers)]
        self.table = torch.full((max_requests, max_pages), -1, **i32)
        self.held = torch.zeros(max_requests, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), num_pages, **i32)
        self.cu = torch.zeros(max_requests + 1, **i32)
        self.positions = torch.full((max_tokens,), -1, **i32)
        self.slots = torch.full((max_tokens,), -1, **i32)
        self.status = torch.zeros(1, **i32)
        self._ctx_len = torch.zeros(max_requests, **i32)
        self.ctx_len = None

    def plan(self, ctx_len, new_len, stream=None) -> Plan:
        """Pages, positions and slots for every request's new_len tokens behind
        its ctx_len cached ones (int32 [max_requests]; both 0 for a free row).  The cache keeps a copy of the
        lengths for the step's attention; the caller may count its own on."""
        if ctx_len.numel() != self.held.numel():
            raise ValueError(f"lengths of all {self.held.numel()} requests are needed")
        made = plan(ctx_len, new_len, self.table, self.held, self.free_pages, self.free_count, self.page_size,
                    cu=self.cu, positions=self.positions, slots=self.slots, status=self.status, stream=stream)
        if stream is None:
            self._ctx_len.copy_(ctx_len.view(-1))
        else:
            with torch.cuda.stream(stream):
                self._ctx_len.copy_(ctx_len.view(-1))
        self.ctx_len = self._ctx_len
        return made

    def append(self, layer: int, qkv, Hq: int, *, q_gamma=None, k_gamma=None, eps: float = 1e-5,
               rope_theta: float = 5e5, out=None, stream=None):
        """The layer's queries, normed and rotated; its keys and values go to their pages."""
        return qk_norm_rope(qkv, Hq, self.Hkv, self.D, self.positions, self.slots, self.kpool[layer],
                            self.vpool[layer], q_gamma=q_gamma, k_gamma=k_gamma, eps=eps, rope_theta=rope_theta,
                            out=out, status=self.status, stream=stream)

    def attention(self, layer: int, q, max_new: int, *, scale: float = None, out=None, stream=None):
        """Attention of the planned step's tokens over the layer's pages."""
        return attention(q, self.kpool[layer], self.vpool[layer], self.table, self.cu, self.ctx_len, max_new,
                         scale=scale, out=out, status=self.status, stream=stream)

    def check(self):
        """Wait for the device; raise if a step's lengths, pages or slots were wrong, whatever stream it ran on
        (and clear the status, before any later step)."""
        torch.cuda.synchronize(self.status.device)
        code = int(self.status.item())
        if code:
            self.status.zero_()
            torch.cuda.synchronize(self.status.device)
            raise L.MkError("PagedCache", code, "the device found a length, page or capacity that does not fit")
