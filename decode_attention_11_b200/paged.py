"""Paged caches and rotary positions: Python binding of the paged part of the tq C ABI.

A pool is a ``Cache`` whose B is the number of pages and whose T_cap is the page size; a ``PageTable``
says which sequence owns which pages.  Everything stays on the device: lists of sequences and pages
are int32 tensors, and a call that finds a bad value in one records it in ``PageTable.status`` (read it
with ``PageTable.check``, which waits for the device).

    pool = tq.Cache.allocate(num_pages, Hkv, page_size, k_bits=4, v_bits=4)
    pt = tq.PageTable.allocate(n_seq, max_pages, num_pages, page_size)
    q, k = tq.rope(q, k, pos)                                     # [N, H, 128], pos int32 [N]
    slots = tq.pages_reserve(pt, seqs, new_tokens, n_slots)       # pages for the new tokens
    tq.paged_quantize(params, k, v, pool, slots)                  # k, v: [N, Hkv, 128]
    out = tq.paged_decode_attn(params, q, pool, pt.table, pt.seq_lens)
    tq.pages_fork(pt, src, dst, [pool]); tq.pages_free(pt, seqs); tq.pages_compact(pt, [pool])
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import (TQ_PAGES_BAD_INDEX, TQ_PAGES_BAD_LENGTH, TQ_PAGES_NO_ROOM, TQ_PAGES_NOT_EMPTY, TQ_PAGES_SHARED,
               TQ_ROPE_HALF, Cache, Params, _Cache, _check, _dtype_code, _PageTable, _ptr, lib)

_STATUS = {TQ_PAGES_NO_ROOM: "not enough free pages", TQ_PAGES_BAD_INDEX: "a number out of range, or listed twice",
           TQ_PAGES_NOT_EMPTY: "fork into a sequence that is not empty", TQ_PAGES_BAD_LENGTH: "bad length",
           TQ_PAGES_SHARED: "growth inside a shared page"}


_INT_MAX = 0x7fffffff  # (ctypes cuts an int to 32 bits without a word; no sequence is longer)


def _elsewhere(device: torch.device, stream) -> bool:
    """Whether the tensors' device or the call's stream is not the current one.  Such a call is made again
    under `_on`, so that what it allocates belongs to that stream; the usual call pays for one test."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {device}")
    if stream is None:
        return device.index != torch.cuda.current_device()
    if stream.device != device:
        raise ValueError(f"stream of {stream.device}, tensors on {device}")
    return True


@contextlib.contextmanager
def _on(device: torch.device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _raw_stream(device: torch.device) -> Optional[int]:
    """Handle of the device's current stream (what torch.cuda.current_stream(device) wraps)."""
    return torch._C._cuda_getCurrentRawStream(device.index) or None


def _int32(t: torch.Tensor, name: str, device: torch.device, dim: int = 1) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != dim or t.device != device:
        raise ValueError(f"{name} must be an int32 tensor of {dim} dimension(s) on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _same_device(device: torch.device, *tensors: Optional[torch.Tensor]) -> None:
    at = device.index
    for t in tensors:
        if t is not None and t.get_device() != (-1 if at is None else at):
            raise ValueError(f"tensors on {t.device} and {device}")


# ---------------------------------------------------------------------------------------- rotary

@functools.lru_cache(maxsize=64)
def _axes_of(sections: Tuple[int, ...]) -> bytes:
    if sum(sections) != 64 or any(s < 0 for s in sections) or not 1 <= len(sections) <= 64:
        raise ValueError(f"sections {sections} must be pair counts of the axes, 64 in all")
    return bytes(a for a, s in enumerate(sections) for _ in range(s))


def _rope_arg(x: Optional[torch.Tensor], out: Optional[torch.Tensor], name: str, N: int):
    """((pointer, strides, heads) of x, its output, the output's pointer)."""
    if x is None:
        return (None, 0, 0, 0), None, None
    if x.dim() != 3:
        raise ValueError(f"{name} must be [N, H, 128]")
    n, H, d = x.shape
    sn, sh, sd = x.stride()
    if n != N or d != 128 or sd != 1:
        raise ValueError(f"{name} must be [N, H, 128] with a contiguous last dim, N = {N}")
    if out is None:
        out = torch.empty_like(x) if sh == 128 and sn == 128 * H else torch.empty(N, H, 128, dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError(f"{name}_out must be contiguous, of the shape and dtype of {name}")
    return (x.data_ptr(), sn, sh, H), out, out.data_ptr()


class _Rope(torch.autograd.Function):
    """rope for inputs that require a gradient: the turn is orthogonal, so the gradient turns back."""

    @staticmethod
    def forward(ctx, q, k, pos, sections, base, style, inverse, axis_of_pair, stream):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(pos)
        ctx.how = sections, base, style, not inverse, axis_of_pair
        return rope(q, k, pos, sections, base, style, inverse, axis_of_pair, stream=stream)

    @staticmethod
    def backward(ctx, *grads):
        pos, = ctx.saved_tensors
        # (gradients come in any strides, a sum's with stride 0)
        g = [x.contiguous() if x is not None and need else None for x, need in zip(grads, ctx.needs_input_grad)]
        g = [x.clone() if x is not None and x.data_ptr() % 16 else x for x in g]
        if g[0] is not None or g[1] is not None:
            g = rope(*g, pos, *ctx.how)
        return (*g, None, None, None, None, None, None, None)


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], pos: torch.Tensor, sections: Sequence[int] = (64,),
         base: float = 10000.0, style: int = TQ_ROPE_HALF, inverse: bool = False,
         axis_of_pair: Optional[Sequence[int]] = None, q_out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions of q [N, Hq, 128] and k [N, Hkv, 128] (either may be None; tq_rope).

    pos: int32 [N], or [axes, N] with one row per axis; sections: how many of the 64 pairs follow each
    axis, in order (or axis_of_pair: the axis of each pair).  inverse=True turns back, and is the
    gradient: d(rope(x))/dx applied to g is rope(g, inverse=True).  Returns (q_out, k_out); q_out = q
    works in place for a contiguous q.  Autograd follows it (not into q_out or k_out)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if torch.is_grad_enabled() and (x.requires_grad or (k is not None and k.requires_grad)):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out / k_out given for an input that requires a gradient")
        return _Rope.apply(q, k, pos, tuple(sections), base, style, inverse,
                           None if axis_of_pair is None else bytes(axis_of_pair), stream)
    device, N, n_axes, pos_stride = x.device, x.shape[0], 1, 0
    if pos.dim() == 2:
        n_axes, n = pos.shape
        pos_stride, step = pos.stride()
    else:
        n, step = (pos.shape[0], pos.stride(0)) if pos.dim() == 1 else (-1, 1)
    if pos.dtype != torch.int32 or n != N or (N > 1 and step != 1):
        raise ValueError(f"pos must be int32 [axes, {N}] with contiguous rows")
    if axis_of_pair is None:
        axes = _axes_of(tuple(sections))
    else:
        axes = bytes(axis_of_pair)
        if len(axes) != 64:
            raise ValueError("axis_of_pair must have 64 entries")
    if q is not None and k is not None and q.dtype != k.dtype:
        raise ValueError("q and k must share their dtype")
    dt = _dtype_code(x)
    _same_device(device, q, k, pos, q_out, k_out)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return rope(q, k, pos, sections, base, style, inverse, axis_of_pair, q_out, k_out)
    qa, q_out, qp = _rope_arg(q, q_out, "q", N)
    ka, k_out, kp = _rope_arg(k, k_out, "k", N)
    _check(lib().tq_rope(*qa, *ka, dt, N, pos.data_ptr(), pos_stride, n_axes, axes, base, style, 1 if inverse else 0, qp, kp,
                         _raw_stream(device)))
    return q_out, k_out


# ---------------------------------------------------------------------------------------- page table

@dataclasses.dataclass
class PageTable:
    """Device arrays that say which sequence owns which pages (tq_page_table)."""

    page_size: int
    table: torch.Tensor     # int32 [n_seq, max_pages], -1: no page
    seq_lens: torch.Tensor  # int32 [n_seq]
    refs: torch.Tensor      # int32 [num_pages], 0: free
    status: torch.Tensor    # int32 [1], sticky TQ_PAGES_* bits

    @classmethod
    def allocate(cls, n_seq: int, max_pages: int, num_pages: int, page_size: int, device="cuda") -> "PageTable":
        i32 = dict(dtype=torch.int32, device=device)
        return cls(page_size, torch.full((n_seq, max_pages), -1, **i32), torch.zeros(n_seq, **i32),
                   torch.zeros(num_pages, **i32), torch.zeros(1, **i32))

    def as_c(self) -> _PageTable:
        d = self.table.device
        _int32(self.table, "table", d, 2), _int32(self.seq_lens, "seq_lens", d)
        _int32(self.refs, "refs", d), _int32(self.status, "status", d)
        if self.seq_lens.shape[0] != self.table.shape[0] or self.status.shape[0] != 1:
            raise ValueError("seq_lens must have one entry per table row, status one entry")
        return _PageTable(self.table.shape[0], self.table.shape[1], self.refs.shape[0], self.page_size,
                          self.table.data_ptr(), self.seq_lens.data_ptr(), self.refs.data_ptr(), self.status.data_ptr())

    def _wait(self) -> None:
        if self.status.is_cuda:
            torch.cuda.synchronize(self.status.device)

    def check(self) -> None:
        """Wait for the device (all its streams); raise ValueError if a call on this table recorded an error,
        and clear it."""
        self._wait()
        bits = int(self.status.item())
        if bits:
            self.status.zero_()
            self._wait()  # a call on another stream must not record before the clearing
            raise ValueError("page table: " + "; ".join(t for b, t in _STATUS.items() if bits & b))


def _caches(caches: Sequence[Cache], device: torch.device):
    for c in caches:
        _same_device(device, c.k_codes, c.k_signs, c.k_norm, c.k_rnorm, c.v_codes, c.v_norm)
    return (_Cache * max(1, len(caches)))(*(c.as_c() for c in caches))


def _workspace(pt: _PageTable, n: int, device: torch.device) -> torch.Tensor:
    return torch.empty(max(16, lib().tq_pages_workspace_size(ctypes.byref(pt), n)), dtype=torch.uint8, device=device)


def pages_reserve(pt: PageTable, seqs: torch.Tensor, new_tokens: torch.Tensor, n_slots: int, stream=None) -> torch.Tensor:
    """Grow sequences seqs[i] by new_tokens[i] tokens (int32 [n] each); returns int32 [n_slots]: the slots
    of the new tokens, sequence after sequence, then -1 (tq_pages_reserve)."""
    device = pt.table.device
    _int32(seqs, "seqs", device), _int32(new_tokens, "new_tokens", device)
    if seqs.shape != new_tokens.shape:
        raise ValueError("seqs and new_tokens must have the same length")
    c = pt.as_c()
    if _elsewhere(device, stream):
        with _on(device, stream):
            return pages_reserve(pt, seqs, new_tokens, n_slots)
    slots = torch.empty(int(n_slots), dtype=torch.int32, device=device)
    ws = _workspace(c, seqs.shape[0], device)
    _check(lib().tq_pages_reserve(ctypes.byref(c), seqs.data_ptr(), new_tokens.data_ptr(), seqs.shape[0],
                                  slots.data_ptr() or None, int(n_slots), ws.data_ptr(), ws.numel(), _raw_stream(device)))
    return slots


def pages_fork(pt: PageTable, src: torch.Tensor, dst: torch.Tensor, caches: Sequence[Cache], stream=None) -> None:
    """Make the empty sequences dst[i] copies of src[i] in every pool (tq_pages_fork)."""
    device = pt.table.device
    _int32(src, "src", device), _int32(dst, "dst", device)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    c, pools = pt.as_c(), _caches(caches, device)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return pages_fork(pt, src, dst, caches)
    ws = _workspace(c, src.shape[0], device)
    _check(lib().tq_pages_fork(ctypes.byref(c), src.data_ptr(), dst.data_ptr(), src.shape[0], pools, len(caches),
                               ws.data_ptr(), ws.numel(), _raw_stream(device)))


def pages_free(pt: PageTable, seqs: torch.Tensor, stream=None) -> None:
    """Release the pages of sequences seqs (int32 [n]; tq_pages_free)."""
    device = pt.table.device
    _int32(seqs, "seqs", device)
    c = pt.as_c()
    if _elsewhere(device, stream):
        with _on(device, stream):
            return pages_free(pt, seqs)
    _check(lib().tq_pages_free(ctypes.byref(c), seqs.data_ptr(), seqs.shape[0], _raw_stream(device)))


def pages_compact(pt: PageTable, caches: Sequence[Cache], stream=None) -> None:
    """Move the pages in use to the lowest page numbers, in every pool (tq_pages_compact)."""
    device = pt.table.device
    c, pools = pt.as_c(), _caches(caches, device)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return pages_compact(pt, caches)
    ws = _workspace(c, 0, device)
    _check(lib().tq_pages_compact(ctypes.byref(c), pools, len(caches), ws.data_ptr(), ws.numel(), _raw_stream(device)))


def pages_copy(caches: Sequence[Cache], src: torch.Tensor, dst: torch.Tensor, status: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """Copy page src[i] to page dst[i] in every pool (int32 [n] each; tq_pages_copy)."""
    device = src.device
    _int32(src, "src", device), _int32(dst, "dst", device)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same length")
    if status is not None:
        _int32(status, "status", device)
        if status.shape[0] != 1:
            raise ValueError("status must have one entry")
    pools = _caches(caches, device)
    if _elsewhere(device, stream):
        with _on(device, stream):
            return pages_copy(caches, src, dst, status)
    _check(lib().tq_pages_copy(pools, len(caches), src.data_ptr(), dst.data_ptr(), src.shape[0], _ptr(status),
                               _raw_stream(device)))


# ---------------------------------------------------------------------------------------- rows

def _slots(slots: torch.Tensor, n: int, device: torch.device) -> torch.Tensor:
    _int32(slots, "slots", device)
    if slots.shape[0] != n:
        raise ValueError(f"slots must have one entry per token ({n})")
    return slots


def paged_quantize(params: Params, k: torch.Tensor, v: torch.Tensor, pool: Cache, slots: torch.Tensor, stream=None) -> None:
    """Compress k, v ([N, Hkv, 128], same strides, last dim contiguous) into the pool's rows at slots
    (int32 [N]; -1: not written; otherwise distinct).  tq_paged_quantize."""
    if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
        raise ValueError("k and v must share shape, strides and dtype")
    if k.dim() != 3 or k.shape[1:] != (pool.Hkv, 128) or (k.numel() and k.stride(2) != 1):
        raise ValueError(f"k must be [N, {pool.Hkv}, 128] with a contiguous last dim")
    device = k.device
    _same_device(device, v, pool.k_codes, params.Pi)
    _slots(slots, k.shape[0], device)
    c, p = pool.as_c(), params.as_c()
    if _elsewhere(device, stream):
        with _on(device, stream):
            return paged_quantize(params, k, v, pool, slots)
    _check(lib().tq_paged_quantize(ctypes.byref(p), k.data_ptr(), v.data_ptr(), _dtype_code(k), k.stride(0),
                                   k.stride(1), k.shape[0], slots.data_ptr(), ctypes.byref(c), _raw_stream(device)))


def paged_read(params: Params, pool: Cache, slots: torch.Tensor, dtype: torch.dtype = torch.float32, stream=None):
    """Rows of the pool at slots (int32 [N]) as values in the rotated basis: (k [N, Hkv, 128], v, signs
    int8 [N, Hkv, 128] of +-1, residual norms [N, Hkv]); signs and norms are None for a pool without
    a sketch; a slot outside the pool reads as zeros.  tq_paged_read."""
    device = slots.device
    _int32(slots, "slots", device)
    _same_device(device, pool.k_codes, params.Pi)
    N, H = slots.shape[0], pool.Hkv
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {dtype}")
    c, p = pool.as_c(), params.as_c()
    if _elsewhere(device, stream):
        with _on(device, stream):
            return paged_read(params, pool, slots, dtype)
    k = torch.empty(N, H, 128, dtype=dtype, device=device)
    v = torch.empty(N, H, 128, dtype=dtype, device=device)
    signs = torch.empty(N, H, 128, dtype=torch.int8, device=device) if pool.qjl_m else None
    rnorm = torch.empty(N, H, dtype=torch.float32, device=device) if pool.qjl_m else None
    _check(lib().tq_paged_read(ctypes.byref(p), ctypes.byref(c), slots.data_ptr(), N, _dtype_code(k), k.data_ptr(),
                               v.data_ptr(), _ptr(signs), _ptr(rnorm), _raw_stream(device)))
    return k, v, signs, rnorm


# ---------------------------------------------------------------------------------------- attention

def paged_decode_workspace_size(B: int, Hq: int, pool: Cache) -> int:
    c = pool.as_c()
    return int(lib().tq_paged_decode_workspace_size(int(B), int(Hq), ctypes.byref(c)))


def paged_decode_attn(params: Params, q: torch.Tensor, pool: Cache, table: torch.Tensor, seq_lens: torch.Tensor,
                      window: int = 0, scale: float = 0.0, out_dtype: torch.dtype = torch.float32,
                      out: Optional[torch.Tensor] = None, return_lse: bool = False,
                      lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of q [B, Hq, 128] over the pages table[b] (int32 [B, max_pages]) and the first seq_lens[b]
    tokens (int32 [B]) of each sequence, or the last `window` of them -> out [B, Hq, 128], or (out, lse)
    with return_lse (lse fp32 [B, Hq], natural log; -inf for an empty sequence).  tq_paged_decode_attn."""
    if q.dim() != 3 or q.shape[2] != 128 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, Hq, 128] tensor")
    B, Hq, _ = q.shape
    device = q.device
    _same_device(device, pool.k_codes, params.Pi, table, out, lse, workspace)
    _int32(seq_lens, "seq_lens", device)
    rows, max_pages = table.shape if table.dim() == 2 else (-1, 0)
    table_stride, step = table.stride() if table.dim() == 2 else (0, 0)
    if table.dtype != torch.int32 or rows != B or (max_pages > 1 and step != 1):
        raise ValueError(f"table must be int32 [{B}, max_pages] with contiguous rows")
    if seq_lens.shape[0] != B:
        raise ValueError(f"seq_lens must have {B} entries")
    c, p = pool.as_c(), params.as_c()
    if _elsewhere(device, stream):
        with _on(device, stream):
            return paged_decode_attn(params, q, pool, table, seq_lens, window, scale, out_dtype, out, return_lse, lse, workspace)
    if out is None:
        out = torch.empty(B, Hq, 128, dtype=out_dtype, device=device)
    elif out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B, Hq, 128] tensor")
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=device) if return_lse else None
    elif lse.shape != (B, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, Hq] tensor")
    if workspace is None:
        workspace = torch.empty(max(16, lib().tq_paged_decode_workspace_size(B, Hq, ctypes.byref(c))), dtype=torch.uint8,
                                device=device)
    _check(lib().tq_paged_decode_attn(
        ctypes.byref(p), q.data_ptr(), _dtype_code(q), B, Hq, ctypes.byref(c), table.data_ptr(),
        table_stride if B > 1 else max(table_stride, max_pages), max_pages, seq_lens.data_ptr(), max(-1, min(window, _INT_MAX)), scale, out.data_ptr(),
        _dtype_code(out), _ptr(lse), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _raw_stream(device)))
    return (out, lse) if return_lse else out
