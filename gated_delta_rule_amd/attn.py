"""Python binding of softmax attention and its paged cache (include/kda_attn.h)
and of the pages' upkeep (include/kda_pages.h).

    o, lse = attn_fwd(q, k, v, cu_seqlens)                        # prompts
    gq, gk, gv = attn_bwd(q, k, v, o, lse, grad_o, cu_seqlens)    # gradients
    kv_append(k, v, k_pages, v_pages, table, lengths)             # new tokens into the cache
    o, lse = attn_paged_fwd(q, k_pages, v_pages, table, lengths)  # their attention over all of it
    ok = kv_resize(table, lengths, refs, new_lengths, page_size)  # grow, roll back, free
    ok = kv_fork(table, lengths, refs, src, dst, pages, page_size)
    table, refs, n_live = kv_compact(table, lengths, refs, pages, page_size)

Arguments are marshalled only; every step runs in the library's HIP kernels.
A serving step: kv_resize to the lengths with the new tokens, kv_append and
attn_paged_fwd in every layer, and after verify_drafts kv_resize to the
lengths without the drafts that fell.  q, k, v and the gradients may be views
of wider token rows, such as the columns of one projection's output; k_pages
and v_pages may be layers of one pool, such as pool[:, layer, 0] and
pool[:, layer, 1] of [n_pages, layers, 2, G, page_size, D].
"""
from __future__ import annotations

import ctypes
import functools

from . import KDA_BF16, KDA_F32, KDAError, _check, _in_dtype, _status, load_library
from .ssm import _NOTHING, _check_rows, _check_shape, _grad_like, _lead, _like, _nbytes, _ptr, _stream, _workspace

__all__ = ["attn_fwd", "attn_bwd", "attn_paged_fwd", "kv_append", "kv_resize", "kv_fork", "kv_compact",
           "attn_bwd_workspace_bytes", "attn_paged_workspace_bytes"]

# Gradients that a backward call makes itself, by their bits in csrc/kda_attn_launch.h.
_FRESH_Q, _FRESH_K, _FRESH_V = 1, 2, 4


def _on(dev):
    """Makes `dev` the current device for the call's launches."""
    import torch
    return _NOTHING if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _of(q, name="q"):
    import torch
    if q.__class__ is torch.Tensor and q.dim() > 2:   # the usual tensors
        if q.dtype is torch.bfloat16:
            return q.device, KDA_BF16
        if q.dtype is torch.float32:
            return q.device, KDA_F32
    if not isinstance(q, torch.Tensor):
        raise KDAError(f"{name} must be a torch.Tensor")
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float32:
        raise KDAError(f"{name} must be bfloat16 or float32, got {q.dtype}")
    if q.dim() < 3:
        raise KDAError(f"{name} must be [..., heads, D]")
    return q.device, _in_dtype(q)


def _scale(scale, D):
    return float(D) ** -0.5 if scale is None else float(scale)


class _Heads:
    """Checked q, k, v of a batch of sequences."""

    __slots__ = ("dev", "dtype", "lead", "n_seqs", "T", "H", "D", "G", "q_tail", "k_tail", "qs", "ks", "vs")

    def __init__(self, q, k, v, cu_seqlens):
        import torch
        self.dev, self.dtype = _of(q)
        self.lead, self.n_seqs, self.T = _lead(q, 2, cu_seqlens, "q", self.dev)
        self.H, self.D = q.shape[-2:]
        if not isinstance(k, torch.Tensor) or k.dim() < 2:
            raise KDAError("k must be [..., G, D]")
        self.G = k.shape[-2]
        self.q_tail, self.k_tail = (self.H, self.D), (self.G, self.D)
        self.qs = _check_rows(q, "q", self.lead, self.q_tail, q.dtype, self.dev)
        self.ks = _check_rows(k, "k", self.lead, self.k_tail, q.dtype, self.dev)
        self.vs = _check_rows(v, "v", self.lead, self.k_tail, q.dtype, self.dev)


def _outputs(q, lead, H, dev, o, lse):
    import torch
    if o is None:
        o = _like(q)
    else:
        _check_shape(o, "o", q.shape, dev, q.dtype)
    if lse is None:
        lse = torch.empty(lead + (H,), dtype=torch.float32, device=dev)
    else:
        _check_shape(lse, "lse", lead + (H,), dev)
    return o, lse


def attn_fwd(q, k, v, cu_seqlens=None, *, scale=None, causal=True, o=None, lse=None):
    """Softmax attention over whole sequences (see kda_attn_fwd in
    include/kda_attn.h).

    q [B, T, H, D], k and v [B, T, G, D] (or packed, without the batch axis,
    with cu_seqlens int32 [n_seqs + 1]), bfloat16 or float32, D 64 or 128, H a
    multiple of G; scale D^-0.5 by default; causal=False: every token sees its
    whole sequence.  Returns (o like q, contiguous; lse [B, T, H] float32).
    Rows of no sequence are not written: in a packed batch that has some,
    outputs that are not given are undefined there.
    """
    lib = load_library()
    a = _Heads(q, k, v, cu_seqlens)
    o, lse = _outputs(q, a.lead, a.H, a.dev, o, lse)
    with _on(a.dev):
        rc = lib.kda_attn_fwd(q.data_ptr(), a.qs, k.data_ptr(), a.ks, v.data_ptr(), a.vs, a.dtype, _ptr(cu_seqlens),
                              a.n_seqs, a.T, a.H, a.G, a.D, _scale(scale, a.D), int(bool(causal)), o.data_ptr(),
                              lse.data_ptr(), _stream(a.dev))
    _status(rc, "kda_attn_fwd")
    return o, lse


@functools.lru_cache(maxsize=256)
def _bwd_bytes(*sizes) -> int:
    return int(load_library().kda_attn_bwd_workspace_bytes(*sizes))


def attn_bwd_workspace_bytes(dtype, n_seqs, T, H, G, D, varlen) -> int:
    """Workspace of attn_bwd for q of this dtype."""
    import torch
    return _bwd_bytes(int(dtype == torch.float32), n_seqs, T, H, G, D, int(bool(varlen)))


def attn_bwd(q, k, v, o, lse, grad_o, cu_seqlens=None, *, scale=None, causal=True, grad_q=None, grad_k=None,
             grad_v=None, workspace=None):
    """Backward pass of attn_fwd (see kda_attn_bwd in include/kda_attn.h).

    Inputs as for the forward call, o and lse what it returned, grad_o like o.
    grad_q, grad_k, grad_v may be given as views of wider rows, like q, k and
    v.  Returns (grad_q, grad_k, grad_v).  In packed batches, rows of no
    sequence keep what they held in tensors that are given and are zero in the
    others.
    """
    lib = load_library()
    a = _Heads(q, k, v, cu_seqlens)
    _check_shape(o, "o", q.shape, a.dev, q.dtype)
    _check_shape(lse, "lse", a.lead + (a.H,), a.dev)
    _check_shape(grad_o, "grad_o", q.shape, a.dev, q.dtype)
    outs, fresh = [], 0
    for name, t, like, tail, bit in (("grad_q", grad_q, q, a.q_tail, _FRESH_Q), ("grad_k", grad_k, k, a.k_tail, _FRESH_K),
                                     ("grad_v", grad_v, v, a.k_tail, _FRESH_V)):
        if t is None:
            t = _grad_like(like, a.n_seqs)
            fresh |= bit
        outs.append((t, _check_rows(t, name, a.lead, tail, q.dtype, a.dev)))
    (gq, gqs), (gk, gks), (gv, gvs) = outs
    ws = _workspace(workspace, _bwd_bytes(a.dtype, a.n_seqs, a.T, a.H, a.G, a.D, int(cu_seqlens is not None)), a.dev)
    with _on(a.dev):
        rc = lib.kda_attn_bwd_fresh(_ptr(q), a.qs, _ptr(k), a.ks, _ptr(v), a.vs, a.dtype, _ptr(cu_seqlens), a.n_seqs,
                                    a.T, a.H, a.G, a.D, _scale(scale, a.D), int(bool(causal)), _ptr(o), _ptr(lse),
                                    _ptr(grad_o), _ptr(gq), gqs, _ptr(gk), gks, _ptr(gv), gvs, _ptr(ws), _nbytes(ws),
                                    _stream(a.dev), fresh)
    _status(rc, "kda_attn_bwd")
    return gq, gk, gv


class _Cache:
    """Checked pages and table of a paged cache."""

    __slots__ = ("n_pages", "G", "page_size", "D", "stride", "n_seqs", "max_pages")

    def __init__(self, k_pages, v_pages, table, lengths, dtype, dev):
        import torch
        tensor, index = torch.Tensor, dev.index
        if k_pages.__class__ is tensor and v_pages.__class__ is tensor and table.__class__ is tensor:   # the usual cache
            shape, st = k_pages.shape, k_pages.stride()
            if len(shape) == 4 and k_pages.dtype is dtype and v_pages.dtype is dtype and v_pages.shape == shape and \
                    v_pages.stride() == st and st[3] == 1 and st[2] == shape[3] and st[1] == shape[2] * st[2] and \
                    k_pages.get_device() == index and v_pages.get_device() == index and table.dtype is torch.int32 and \
                    table.get_device() == index and table.dim() == 2 and table.is_contiguous():
                self.n_pages, self.G, self.page_size, self.D = shape
                self.stride = st[0]
                self.n_seqs, self.max_pages = table.shape
                _check_shape(lengths, "lengths", (self.n_seqs,), dev, torch.int32)
                return
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(t, torch.Tensor) or t.dim() != 4:
                raise KDAError(f"{name} must be [n_pages, G, page_size, D]")
            if not t.is_cuda:
                raise KDAError(f"{name} must be a device tensor")
            if t.device != dev:
                raise KDAError(f"{name} is on {t.device}, expected {dev}")
            if t.dtype != dtype:
                raise KDAError(f"{name} must be {dtype}, got {t.dtype}")
            if t.numel() and not t[0].is_contiguous():
                raise KDAError(f"{name} must be contiguous within a page")
        if k_pages.shape != v_pages.shape:
            raise KDAError("k_pages and v_pages must have the same shape")
        self.n_pages, self.G, self.page_size, self.D = k_pages.shape
        if self.n_pages > 1 and k_pages.stride(0) != v_pages.stride(0):
            raise KDAError("k_pages and v_pages must have the same page stride")
        self.stride = k_pages.stride(0) if self.n_pages > 1 else self.G * self.page_size * self.D
        _check(table, "table", torch.int32, dev)
        if table.dim() != 2:
            raise KDAError("table must be [n_seqs, max_pages]")
        self.n_seqs, self.max_pages = table.shape
        _check_shape(lengths, "lengths", (self.n_seqs,), dev, torch.int32)


def _requests(c, n_seqs):
    if n_seqs != c.n_seqs:
        raise KDAError(f"table holds {c.n_seqs} requests, the batch {n_seqs}")


def kv_append(k, v, k_pages, v_pages, table, lengths, cu_seqlens=None):
    """New tokens' keys and values into a paged cache (see kda_kv_append in
    include/kda_attn.h).

    k, v [B, T, G, D] (or packed [T, G, D] with cu_seqlens int32 [B + 1]);
    k_pages, v_pages [n_pages, G, page_size, D], page_size 16 to 256, updated in
    place; table int32 [B, max_pages]; lengths int32 [B], the new tokens
    included: they take the last places of their requests.
    """
    lib = load_library()
    dev, dt = _of(k, "k")
    lead, n_seqs, T = _lead(k, 2, cu_seqlens, "k", dev)
    c = _Cache(k_pages, v_pages, table, lengths, k.dtype, dev)
    _requests(c, n_seqs)
    ks = _check_rows(k, "k", lead, (c.G, c.D), k.dtype, dev)
    vs = _check_rows(v, "v", lead, (c.G, c.D), k.dtype, dev)
    with _on(dev):
        rc = lib.kda_kv_append(k.data_ptr(), ks, v.data_ptr(), vs, dt, k_pages.data_ptr(), v_pages.data_ptr(), c.stride,
                               c.n_pages, c.page_size, table.data_ptr(), c.max_pages, lengths.data_ptr(),
                               _ptr(cu_seqlens), n_seqs, T, c.G, c.D, _stream(dev))
    _status(rc, "kda_kv_append")


@functools.lru_cache(maxsize=256)
def _paged_bytes(*sizes) -> int:
    return int(load_library().kda_attn_paged_workspace_bytes(*sizes))


def attn_paged_workspace_bytes(dtype, n_seqs, T, H, G, D, page_size, max_pages, varlen) -> int:
    """Workspace of attn_paged_fwd for q of this dtype."""
    import torch
    return _paged_bytes(int(dtype == torch.float32), n_seqs, T, H, G, D, page_size, max_pages, int(bool(varlen)))


def attn_paged_fwd(q, k_pages, v_pages, table, lengths, cu_seqlens=None, *, scale=None, o=None, lse=None,
                   workspace=None):
    """Attention of the last tokens of requests over all of their tokens up to
    their own, from a paged cache that holds them all (see kda_attn_paged_fwd in
    include/kda_attn.h).

    q [B, T, H, D] (or packed [T, H, D] with cu_seqlens int32 [B + 1]); cache
    arguments as for kv_append.  Returns (o like q, contiguous; lse [B, T, H]
    float32).  Rows of no request are not written: in a packed batch that has
    some, outputs that are not given are undefined there.
    """
    lib = load_library()
    dev, dt = _of(q)
    lead, n_seqs, T = _lead(q, 2, cu_seqlens, "q", dev)
    c = _Cache(k_pages, v_pages, table, lengths, q.dtype, dev)
    _requests(c, n_seqs)
    H, D = q.shape[-2:]
    if D != c.D:
        raise KDAError(f"q must have head dimension {c.D}, got {D}")
    qs = _check_rows(q, "q", lead, (H, D), q.dtype, dev)
    o, lse = _outputs(q, lead, H, dev, o, lse)
    ws = _workspace(workspace, _paged_bytes(dt, n_seqs, T, H, c.G, D, c.page_size, c.max_pages,
                                            int(cu_seqlens is not None)), dev)
    with _on(dev):
        rc = lib.kda_attn_paged_fwd(q.data_ptr(), qs, dt, k_pages.data_ptr(), v_pages.data_ptr(), c.stride, c.n_pages,
                                    c.page_size, table.data_ptr(), c.max_pages, lengths.data_ptr(), _ptr(cu_seqlens),
                                    n_seqs, T, H, c.G, D, _scale(scale, D), o.data_ptr(), lse.data_ptr(), _ptr(ws),
                                    _nbytes(ws), _stream(dev))
    _status(rc, "kda_attn_paged_fwd")
    return o, lse


@functools.lru_cache(maxsize=256)
def _page_layout(layouts):
    """Bytes and strides of pages, as arrays for the library, from each tensor's
    (shape, strides, element size)."""
    size, step = [], []
    for shape, strides, width in layouts:
        elements = 1
        for n, s in zip(reversed(shape[1:]), reversed(strides[1:])):
            if n > 1 and s != elements:
                raise KDAError("pages must be contiguous within a page")
            elements *= n
        size.append(elements * width)
        step.append(strides[0] * width)
    n = len(layouts)
    return (ctypes.c_int64 * n)(*size), (ctypes.c_int64 * n)(*step)


class _Pages:
    """Checked table, lengths and refs."""

    __slots__ = ("dev", "n_slots", "max_pages", "n_pages")

    def __init__(self, table, lengths, refs):
        import torch
        tensor, i32 = torch.Tensor, torch.int32
        if table.__class__ is tensor and lengths.__class__ is tensor and refs.__class__ is tensor and table.is_cuda:   # the usual ones
            i = table.get_device()
            if table.dtype is i32 and lengths.dtype is i32 and refs.dtype is i32 and lengths.get_device() == i and \
                    refs.get_device() == i and table.dim() == 2 and lengths.dim() == 1 and refs.dim() == 1 and \
                    lengths.shape[0] == table.shape[0] and table.is_contiguous() and lengths.is_contiguous() and \
                    refs.is_contiguous():
                self.dev = table.device
                self.n_slots, self.max_pages = table.shape
                self.n_pages = refs.shape[0]
                return
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise KDAError("table must be [n_slots, max_pages]")
        self.dev = table.device
        _check(table, "table", torch.int32, self.dev)
        self.n_slots, self.max_pages = table.shape
        _check_shape(lengths, "lengths", (self.n_slots,), self.dev, torch.int32)
        _check(refs, "refs", torch.int32, self.dev)
        if refs.dim() != 1:
            raise KDAError("refs must be [n_pages]")
        self.n_pages = refs.shape[0]

    def data(self, pages):
        """(pointers, bytes, strides, count) of the tensors that hold the pages."""
        import torch
        tensors = (pages,) if isinstance(pages, torch.Tensor) else tuple(pages)
        index, layouts = self.dev.index, []
        for t in tensors:
            if not isinstance(t, torch.Tensor) or t.dim() < 2:
                raise KDAError("pages must be tensors [n_pages, ...]")
            if not t.is_cuda or t.get_device() != index:
                raise KDAError(f"pages must be on {self.dev}")
            if t.shape[0] != self.n_pages:
                raise KDAError(f"pages must have {self.n_pages} pages, got {t.shape[0]}")
            layouts.append((t.shape, t.stride(), t.element_size()))
        n = len(tensors)
        return ((ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]),) + _page_layout(tuple(layouts)) + (n,)


def kv_resize(table, lengths, refs, new_lengths, page_size):
    """Sets the length of every slot: grows it with free pages or gives up
    pages that it no longer needs; 0 frees it (see kda_kv_resize in
    include/kda_pages.h).

    table int32 [n_slots, max_pages], lengths int32 [n_slots], refs int32
    [n_pages] (holders of each page), all updated in place; new_lengths int32
    [n_slots].  Returns ok int32 [n_slots]: 0 where no pages were left, and the
    slot is as it was.  A slot that is cut back into a page shared with a branch
    still shares it: kv_fork it to another slot before appending.
    """
    import torch
    lib = load_library()
    a = _Pages(table, lengths, refs)
    _check_shape(new_lengths, "new_lengths", (a.n_slots,), a.dev, torch.int32)
    ok = _like(lengths)
    with _on(a.dev):
        rc = lib.kda_kv_resize(_ptr(table), _ptr(lengths), _ptr(refs), _ptr(new_lengths), _ptr(ok), a.n_slots,
                               a.max_pages, a.n_pages, page_size, _stream(a.dev))
    _status(rc, "kda_kv_resize")
    return ok


@functools.lru_cache(maxsize=256)
def _fork_bytes(*sizes) -> int:
    return int(load_library().kda_kv_fork_workspace_bytes(*sizes))


def kv_fork(table, lengths, refs, src, dst, pages, page_size, *, workspace=None):
    """Makes slots dst branches of slots src, all at once: they share src's full
    pages and get a copy of an open last one (see kda_kv_fork in
    include/kda_pages.h).

    table, lengths, refs as for kv_resize, updated in place; src, dst int32
    [n]; pages the tensor [n_pages, ...], or up to 16 of them, that hold the
    pages' data.  Returns ok int32 [n]: 0 where dst stays as it was.  With too
    few free pages only pairs that copy one are refused, the later ones.
    """
    import torch
    lib = load_library()
    a = _Pages(table, lengths, refs)
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise KDAError("src must be [n]")
    _check_shape(src, "src", src.shape, a.dev, torch.int32)
    _check_shape(dst, "dst", src.shape, a.dev, torch.int32)
    ptrs, size, step, count = a.data(pages)
    ok = _like(src)
    n = src.shape[0]
    ws = _workspace(workspace, _fork_bytes(n, a.n_slots, a.max_pages), a.dev)
    with _on(a.dev):
        rc = lib.kda_kv_fork(_ptr(table), _ptr(lengths), _ptr(refs), _ptr(src), _ptr(dst), _ptr(ok), n, a.n_slots,
                             a.max_pages, a.n_pages, page_size, ptrs, size, step, count, _ptr(ws), _nbytes(ws),
                             _stream(a.dev))
    _status(rc, "kda_kv_fork")
    return ok


def kv_compact(table, lengths, refs, pages, page_size, *, table_out=None, refs_out=None, workspace=None):
    """Moves the pages in use to the lowest numbers (see kda_kv_compact in
    include/kda_pages.h).

    Arguments as for kv_fork; the pages' data moves in place.  Returns (table,
    refs, n_live int32 [1]), new tensors or table_out and refs_out, which may be
    table and refs themselves.
    """
    import torch
    lib = load_library()
    a = _Pages(table, lengths, refs)
    ptrs, size, step, count = a.data(pages)
    if table_out is None:
        table_out = _like(table)
    else:
        _check_shape(table_out, "table_out", table.shape, a.dev, torch.int32)
    if refs_out is None:
        refs_out = _like(refs)
    else:
        _check_shape(refs_out, "refs_out", refs.shape, a.dev, torch.int32)
    n_live = torch.empty((1,), dtype=torch.int32, device=a.dev)
    ws = _workspace(workspace, int(lib.kda_kv_compact_workspace_bytes(a.n_pages)), a.dev)
    with _on(a.dev):
        rc = lib.kda_kv_compact(_ptr(table), _ptr(lengths), _ptr(refs), _ptr(table_out), _ptr(refs_out), _ptr(n_live),
                                a.n_slots, a.max_pages, a.n_pages, page_size, ptrs, size, step, count, _ptr(ws),
                                _nbytes(ws), _stream(a.dev))
    _status(rc, "kda_kv_compact")
    return table_out, refs_out, n_live
