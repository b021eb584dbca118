"""A paged KV cache: block tables and slot maps, per-head norms with rotation
and page stores, and attention of new tokens over the pages (the operators
mk_paged_plan, mk_qk_norm_rope and mk_paged_attention of include/mk.h).

The functions take PyTorch tensors on one CUDA device and enqueue on that
device's current stream, or on ``stream``; nothing synchronises.  Lengths,
tables and maps are int32 tensors that the GPU reads; what is wrong with
their values is reported in ``status`` (an int32 device tensor, zeroed by the
caller, that receives the first MK_DEV_* code).  ``PagedCache`` holds a
cache's pools, tables and free pages and runs the operators on them.
"""
from __future__ import annotations

from functools import lru_cache
from typing import NamedTuple

import torch

from . import _lib as L

_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle, without a Stream object
_current_device = torch.cuda.current_device
_alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc     # scratch of one call from PyTorch's allocator, ordered by the
_free = torch._C._cuda_cudaCachingAllocator_raw_delete     # stream as a tensor's memory is, without the tensor


def on_stream(fn, dev: int, stream, args, kw):
    """Call ``fn`` with ``stream`` current (its device too), or with device ``dev`` current."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    with torch.cuda.device(dev):
        return fn(*args, **kw)


def device_of(t, name) -> int:
    """Index of the CUDA device of an operator's first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def int32_ptr(t, name, n, dev):
    """Address of a contiguous int32 tensor of at least n elements."""
    if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} elements on cuda:{dev}")
    return t.data_ptr()


def _table(table, B, dev):
    """(address, pages per request) of the block tables of at least B requests."""
    if table.dtype is not _I32 or table.get_device() != dev or not table.is_contiguous() or table.dim() != 2 \
            or table.shape[0] < B:
        raise ValueError(f"table must be contiguous int32 [{B} or more requests, pages] on cuda:{dev}")
    return table.data_ptr(), table.shape[1]


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
    ``count_out`` are given.  ``positions`` and ``slots`` (or ``max_tokens``)
    set how many new tokens the step can have."""
    dev = device_of(ctx_len, "ctx_len")
    if stream is not None or dev != _current_device():
        return on_stream(plan, dev, stream, (ctx_len, new_len, table, held, free_pages, free_count, page_size),
                         dict(cu=cu, positions=positions, slots=slots, max_tokens=max_tokens, held_out=held_out,
                              count_out=count_out, status=status))
    B = ctx_len.numel()
    tab, max_pages = _table(table, B, dev)
    if positions is None or slots is None:
        if max_tokens is None:
            raise ValueError("give positions and slots, or max_tokens")
        positions = torch.empty(max_tokens, dtype=_I32, device=ctx_len.device) if positions is None else positions
        slots = torch.empty(max_tokens, dtype=_I32, device=ctx_len.device) if slots is None else slots
    if cu is None:
        cu = torch.empty(B + 1, dtype=_I32, device=ctx_len.device)
    n = positions.numel()
    h, c = int32_ptr(held, "held", B, dev), int32_ptr(free_count, "free_count", 1, dev)
    L.mk_paged_plan(_raw_stream(dev), B, page_size, max_pages, free_pages.numel(), n,
                    int32_ptr(ctx_len, "ctx_len", B, dev), int32_ptr(new_len, "new_len", B, dev), tab, h,
                    h if held_out is None else int32_ptr(held_out, "held_out", B, dev),
                    int32_ptr(free_pages, "free_pages", 1, dev), c,
                    c if count_out is None else int32_ptr(count_out, "count_out", 1, dev),
                    int32_ptr(cu, "cu", B + 1, dev), int32_ptr(positions, "positions", n, dev),
                    int32_ptr(slots, "slots", n, dev), 0 if status is None else int32_ptr(status, "status", 1, dev))
    return Plan(cu, positions, slots)


def _pools(kpool, vpool, dev):
    """The pools' common shape [num_pages, Hkv, page_size, D]."""
    s = kpool.shape
    if (len(s) != 4 or vpool.shape != s or kpool.dtype is not _BF16 or vpool.dtype is not _BF16
            or not kpool.is_contiguous() or not vpool.is_contiguous() or kpool.get_device() != dev
            or vpool.get_device() != dev):
        raise ValueError(f"kpool and vpool must be contiguous bf16 [num_pages, Hkv, page_size, D] on cuda:{dev}")
    return s


def _rows(t, name, N, Hq, D, dev):
    """Elements between the rows of bf16 [N, Hq, D], which may lie apart."""
    if t.dtype is not _BF16 or t.get_device() != dev or t.shape != (N, Hq, D):
        raise ValueError(f"{name} must be bf16 [{N}, {Hq}, {D}] on cuda:{dev}")
    if t.is_contiguous():
        return Hq * D
    row, head, one = t.stride()
    if (D > 1 and one != 1) or (Hq > 1 and head != D):
        raise ValueError(f"each row of {name} must be contiguous")
    return row if N > 1 else Hq * D


def qk_norm_rope(qkv, Hq: int, Hkv: int, D: int, positions, slots, kpool, vpool, *, q_gamma=None, k_gamma=None,
                 eps: float = 1e-5, rope_theta: float = 5e5, out=None, status=None, stream=None):
    """RMS norms of queries and keys for each head (none where its gain is
    None), the rotate-half rotary embedding at ``positions``, and the stores
    of keys and values at ``slots`` (mk_qk_norm_rope).  qkv f32 or bf16
    [N, (Hq + 2 Hkv) D], rows may lie apart; returns the queries, bf16
    [N, Hq, D] (``out`` if given).  Rows with a negative position are left
    out; ``out`` keeps what it had there (a fresh one holds anything)."""
    dev = device_of(qkv, "qkv")
    if stream is not None or dev != _current_device():
        return on_stream(qk_norm_rope, dev, stream, (qkv, Hq, Hkv, D, positions, slots, kpool, vpool),
                         dict(q_gamma=q_gamma, k_gamma=k_gamma, eps=eps, rope_theta=rope_theta, out=out, status=status))
    width = (Hq + 2 * Hkv) * D
    dt = qkv.dtype
    if (dt is not _F32 and dt is not _BF16) or qkv.dim() != 2 or qkv.shape[1] != width or qkv.stride(1) != 1:
        raise ValueError(f"qkv must be f32 or bf16 [N, {width}] with contiguous rows")
    N = qkv.shape[0]
    num_pages, kv, page, d = _pools(kpool, vpool, dev)
    if kv != Hkv or d != D:
        raise ValueError(f"the pools have {kv} heads of {d}, the call {Hkv} of {D}")
    if out is None:
        out = torch.empty(N, Hq, D, dtype=_BF16, device=qkv.device)
    ld_q = _rows(out, "out", N, Hq, D, dev)
    if q_gamma is not None and (q_gamma.dtype is not _BF16 or q_gamma.numel() != D or not q_gamma.is_contiguous()
                                or q_gamma.get_device() != dev):
        raise ValueError(f"q_gamma must be bf16 [{D}] on cuda:{dev}")
    if k_gamma is not None and (k_gamma.dtype is not _BF16 or k_gamma.numel() != D or not k_gamma.is_contiguous()
                                or k_gamma.get_device() != dev):
        raise ValueError(f"k_gamma must be bf16 [{D}] on cuda:{dev}")
    if N == 0:
        return out
    L.mk_qk_norm_rope(_raw_stream(dev), N, Hq, Hkv, D, qkv.data_ptr(), L.MK_F32 if dt is _F32 else L.MK_BF16,
                      qkv.stride(0) if N > 1 else width, 0 if q_gamma is None else q_gamma.data_ptr(),
                      0 if k_gamma is None else k_gamma.data_ptr(), eps, rope_theta,
                      int32_ptr(positions, "positions", N, dev), int32_ptr(slots, "slots", N, dev), out.data_ptr(),
                      ld_q, kpool.data_ptr(), vpool.data_ptr(), num_pages, page,
                      0 if status is None else int32_ptr(status, "status", 1, dev))
    return out


@lru_cache(maxsize=None)
def _workspace_bytes(dev: int, max_new: int, Hq: int, Hkv: int, D: int) -> int:
    with torch.cuda.device(dev):
        return L.mk_paged_attention_workspace(max_new, Hq, Hkv, D)


def attention_workspace(max_new: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    """A workspace for ``attention`` with these sizes.  Calls that share one
    must not overlap: run them on one stream."""
    dev = torch.device(device)
    index = dev.index if dev.index is not None else _current_device()
    return torch.empty(_workspace_bytes(index, max_new, Hq, Hkv, D), dtype=_U8, device=dev)


def attention(q, kpool, vpool, table, cu, ctx_len, max_new: int, *, scale: float = None, out=None, workspace=None,
              status=None, stream=None):
    """Attention of the requests' new tokens over their pages, causal among
    the new ones (mk_paged_attention).  q bf16 [N, Hq, D] (rows may lie
    apart), row cu[b] + t is token t of request b, which sees the keys at
    positions 0 .. ctx_len[b] + t of the pages table[b]; no request has more
    than ``max_new`` new tokens.  Returns ``out`` bf16 [N, Hq, D]; rows of no
    request keep what it had (a fresh one holds anything).  Without a
    ``workspace`` one is taken from PyTorch's allocator for the call."""
    dev = device_of(q, "q")
    if stream is not None or dev != _current_device():
        return on_stream(attention, dev, stream, (q, kpool, vpool, table, cu, ctx_len, max_new),
                         dict(scale=scale, out=out, workspace=workspace, status=status))
    num_pages, Hkv, page, D = _pools(kpool, vpool, dev)
    if q.dim() != 3:
        raise ValueError("q must be bf16 [N, Hq, D]")
    N, Hq, _ = q.shape
    ld_q = _rows(q, "q", N, Hq, D, dev)
    if out is None:
        out = torch.empty(N, Hq, D, dtype=_BF16, device=q.device)
    ld_out = _rows(out, "out", N, Hq, D, dev)
    B = ctx_len.numel()
    tab, max_pages = _table(table, B, dev)
    if N == 0 or B == 0:
        return out
    stream = _raw_stream(dev)
    scratch = 0
    if workspace is None:
        size = _workspace_bytes(dev, max_new, Hq, Hkv, D)
        work = scratch = _alloc(size, stream)
    elif workspace.is_contiguous() and workspace.get_device() == dev:
        work, size = workspace.data_ptr(), workspace.nbytes
    else:
        raise ValueError(f"workspace must be contiguous on cuda:{dev}")
    try:
        L.mk_paged_attention(stream, B, N, max_new, Hq, Hkv, D, q.data_ptr(), ld_q, kpool.data_ptr(), vpool.data_ptr(),
                             num_pages, page, tab, max_pages, int32_ptr(cu, "cu", B + 1, dev),
                             int32_ptr(ctx_len, "ctx_len", B, dev), D ** -0.5 if scale is None else scale,
                             out.data_ptr(), ld_out, work, size,
                             0 if status is None else int32_ptr(status, "status", 1, dev))
    finally:
        if scratch:
            _free(scratch)
    return out


class PagedCache:
    """The KV cache of ``layers`` layers in pages, for up to ``max_requests``
    requests and ``max_tokens`` new tokens a step.  Per step: ``plan`` with
    the requests' lengths, then per layer ``append`` (norms, rotation, page
    stores) and ``attention``.  A request that ends, or whose drafts were
    rejected, gives its pages back through the next plan's lengths."""

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
        self.ctx_len = None

    def plan(self, ctx_len, new_len, stream=None) -> Plan:
        """Pages, positions and slots for every request's new_len tokens behind
        its ctx_len cached ones (int32 [max_requests]; both 0 for a free row)."""
        if ctx_len.numel() != self.held.numel():
            raise ValueError(f"lengths of all {self.held.numel()} requests are needed")
        self.ctx_len = ctx_len
        return plan(ctx_len, new_len, self.table, self.held, self.free_pages, self.free_count, self.page_size,
                    cu=self.cu, positions=self.positions, slots=self.slots, status=self.status, stream=stream)

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
        """Synchronise; raise if a step's lengths, pages or slots were wrong (and clear the status)."""
        code = int(self.status.item())
        if code:
            self.status.zero_()
            raise L.MkError("PagedCache", code, "the device found a length, page or capacity that does not fit")
