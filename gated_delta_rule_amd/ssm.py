"""Python binding of the state space scan and its short convolution
(include/kda_ssm.h) and of the draft verification (include/kda_spec.h).

    y = ssm_conv_fwd(xbc, w, bias, cache, cu_seqlens)             # prompts, cache in place
    y, S_T = ssm_chunk_fwd(x, dt, A, B, C, D, S0, cu_seqlens)     # prompts
    y = ssm_conv_step(xbc, w, bias, cache, replay=, n_replay=)    # up to 64 tokens per request
    y = ssm_recurrent_fwd(x, dt, A, B, C, S, D, replay=, n_replay=)
    n_accepted, tokens = verify_drafts(p_target, drafts, u, u_next, p_draft)
    ssm_conv_bwd, ssm_chunk_bwd                                   # gradients

Arguments are marshalled only; every step runs in the library's HIP kernels.
x, B, C and the gradients may be views of wider token rows, such as the
channels of one convolution's output:

    x, B, C = y.split([H * P, G * N, G * N], -1), each unflattened to
    [..., H, P] and [..., G, N]
"""
from __future__ import annotations

import contextlib
import math

from . import KDA_BF16, KDA_F32, KDAError, _check, _in_dtype, _status, load_library

__all__ = ["ssm_conv_fwd", "ssm_conv_step", "ssm_conv_bwd", "ssm_chunk_fwd", "ssm_chunk_bwd",
           "ssm_recurrent_fwd", "ssm_chunk_fwd_workspace_bytes", "ssm_chunk_bwd_workspace_bytes",
           "verify_drafts"]

_NOTHING = contextlib.nullcontext()


def _on(dev):
    """Makes `dev` the current device for the call's launches."""
    import torch
    return _NOTHING if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(dev):
    """The current stream of `dev` (torch.cuda.current_stream builds an object for it, 2 us)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _of(x):
    """Device and element type of a call's x."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise KDAError("x must be a torch.Tensor")
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float32:
        raise KDAError(f"x must be bfloat16 or float32, got {x.dtype}")
    return x.device, _in_dtype(x)


def _check_rows(t, name, lead, tail, dtype, dev):
    """A tensor [*lead, *tail] whose rows (the tail) are contiguous and evenly
    spaced over the leading axes; returns the row stride in elements."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise KDAError(f"{name} must be a torch.Tensor")
    if t.get_device() == dev.index and t.dtype is dtype and t.shape == lead + tail:   # the usual rows
        if t.is_contiguous():
            return math.prod(tail)
        st, nl = t.stride(), len(lead)
        if lead[-1] > 1 and st[-1] == 1 and (len(tail) == 1 or tail[0] == 1 or st[-2] == tail[1]) and \
                (nl == 1 or lead[0] == 1 or st[0] == lead[1] * st[1]) and t.numel():
            return st[nl - 1]
    if not t.is_cuda:
        raise KDAError(f"{name} must be a device tensor")
    if t.device != dev:
        raise KDAError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise KDAError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(lead) + tuple(tail):
        raise KDAError(f"{name} must be {tuple(lead) + tuple(tail)}, got {tuple(t.shape)}")
    width, strides, nl = 1, t.stride(), len(lead)
    if t.numel() == 0:
        for n in tail:
            width *= n
        return width
    for n, s in zip(reversed(tail), reversed(strides[nl:])):
        if n != 1 and s != width:
            raise KDAError(f"{name} must be contiguous within a token row")
        width *= n
    stride = None
    rows = 1
    for n, s in zip(reversed(lead), reversed(strides[:nl])):
        if n != 1:
            if stride is None:
                if s % rows:
                    raise KDAError(f"{name} must have evenly spaced token rows")
                stride = s // rows
            if s != stride * rows:
                raise KDAError(f"{name} must have evenly spaced token rows")
        rows *= n
    return width if stride is None else stride


def _lead(x, tail_dims, cu_seqlens, name, dev):
    """Leading shape, number of sequences and T of a batch."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise KDAError(f"{name} must be a torch.Tensor")
    lead = tuple(x.shape[:x.dim() - tail_dims])
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise KDAError("cu_seqlens must be [n_seqs + 1]")
        if len(lead) == 2 and lead[0] == 1 or len(lead) == 1:
            return lead, cu_seqlens.numel() - 1, lead[-1]
        raise KDAError(f"packed {name} must have one token axis (a leading batch of 1 is allowed)")
    if len(lead) != 2:
        raise KDAError(f"{name} must have batch and token axes without cu_seqlens")
    return lead, lead[0], lead[1]


def _check_shape(t, name, shape, dev, dtype=None):
    import torch
    dtype = dtype or torch.float32
    if t.__class__ is torch.Tensor and t.get_device() == dev.index and t.dtype is dtype and t.shape == shape and \
            t.is_contiguous():
        return
    _check(t, name, dtype, dev)
    if tuple(t.shape) != tuple(shape):
        raise KDAError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _workspace(workspace, need, dev):
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check(workspace, "workspace", None, dev)
    return workspace


def _like(t):
    """An uninitialised contiguous tensor like t (half the time of torch.empty)."""
    import torch
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# Outputs that a backward call makes itself, by their bits in csrc/kda_ssm_launch.h.
_FRESH_X, _FRESH_B, _FRESH_C, _FRESH_DT = 1, 2, 4, 8


def _grad_like(t, n_seqs):
    """Like _like, for the gradient of token rows: the kernels write every row
    of a batch that has a sequence at all."""
    import torch
    return _like(t) if n_seqs else torch.zeros_like(t, memory_format=torch.contiguous_format)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _conv_args(x, w, bias):
    import torch
    dev, dt = _of(x)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise KDAError("w must be [channels, width]")
    _check(w, "w", torch.float32, dev)
    channels, width = w.shape
    if bias is not None:
        _check_shape(bias, "bias", (channels,), dev)
    return dev, dt, channels, width


def ssm_conv_fwd(x, w, bias=None, cache=None, cu_seqlens=None, *, activation=True, y=None):
    """Short causal depthwise convolution with SiLU (see kda_ssm_conv_fwd in
    include/kda_ssm.h).

    x [B, T, channels] (or packed [T, channels] with cu_seqlens), bfloat16 or
    float32; w [channels, width] float32; bias [channels] or None; cache
    [n_seqs, width - 1, channels] float32, updated in place, or None.
    activation=False leaves out the SiLU.  Returns y like x, contiguous.  Rows
    of no sequence are not written: in a packed batch that has some, a y that
    is not given is undefined there.
    """
    import torch
    lib = load_library()
    dev, dt, channels, width = _conv_args(x, w, bias)
    lead, n_seqs, T = _lead(x, 1, cu_seqlens, "x", dev)
    xs = _check_rows(x, "x", lead, (channels,), x.dtype, dev)
    if cache is not None:
        _check_shape(cache, "cache", (n_seqs, width - 1, channels), dev)
    if y is None:
        y = _like(x)
    else:
        _check_shape(y, "y", x.shape, dev, x.dtype)
    with _on(dev):
        rc = lib.kda_ssm_conv_fwd(_ptr(x), xs, dt, _ptr(w), _ptr(bias), _ptr(cache), _ptr(cu_seqlens),
                                  n_seqs, T, channels, width, int(bool(activation)), _ptr(y), _stream(dev))
    _status(rc, "kda_ssm_conv_fwd")
    return y


def ssm_conv_step(x, w, bias, cache, *, replay=None, n_replay=None, commit=True, activation=True, y=None):
    """The convolution of up to 64 new tokens per request (see
    kda_ssm_conv_step in include/kda_ssm.h).

    x [B, T, channels]; cache [B, width - 1, channels] float32, updated in
    place: it takes in the first n_replay[b] (int32 [B] on the device; None:
    all) tokens of replay [B, Tr, channels] and, with commit=True, the new
    tokens.  Returns y [B, T, channels].
    """
    import torch
    lib = load_library()
    dev, dt, channels, width = _conv_args(x, w, bias)
    lead, B, T = _lead(x, 1, None, "x", dev)
    xs = _check_rows(x, "x", lead, (channels,), x.dtype, dev)
    _check_shape(cache, "cache", (B, width - 1, channels), dev)
    Tr, rs = 0, channels
    if replay is not None:
        rlead, Br, Tr = _lead(replay, 1, None, "replay", dev)
        if Br != B:
            raise KDAError("replay and x must have the same number of requests")
        rs = _check_rows(replay, "replay", rlead, (channels,), x.dtype, dev)
    if n_replay is not None:
        _check_shape(n_replay, "n_replay", (B,), dev, torch.int32)
    if y is None:
        y = _like(x)
    else:
        _check_shape(y, "y", (B, T, channels), dev, x.dtype)
    with _on(dev):
        rc = lib.kda_ssm_conv_step(_ptr(x), xs, dt, _ptr(w), _ptr(bias), _ptr(cache), _ptr(replay), rs,
                                   _ptr(n_replay), B, T, Tr, channels, width, int(bool(activation)),
                                   int(bool(commit)), _ptr(y), _stream(dev))
    _status(rc, "kda_ssm_conv_step")
    return y


def ssm_conv_bwd(x, w, bias, grad_y, cache=None, cu_seqlens=None, *, activation=True, workspace=None):
    """Backward pass of ssm_conv_fwd (see kda_ssm_conv_bwd in
    include/kda_ssm.h).  `cache` is the one from before the forward call.
    Returns (grad_x in x's dtype, grad_w, grad_bias, grad_cache); grad_bias
    and grad_cache are None where bias and cache are.  In packed batches
    grad_x is zero in rows of no sequence.
    """
    import torch
    lib = load_library()
    dev, dt, channels, width = _conv_args(x, w, bias)
    lead, n_seqs, T = _lead(x, 1, cu_seqlens, "x", dev)
    xs = _check_rows(x, "x", lead, (channels,), x.dtype, dev)
    gs = _check_rows(grad_y, "grad_y", lead, (channels,), x.dtype, dev)
    if cache is not None:
        _check_shape(cache, "cache", (n_seqs, width - 1, channels), dev)
    gx, gw = _grad_like(x, n_seqs), _like(w)
    gb = None if bias is None else _like(bias)
    gc = None if cache is None else _like(cache)
    rows = T if cu_seqlens is not None else n_seqs * T
    ws = _workspace(workspace, int(lib.kda_ssm_conv_bwd_workspace_bytes(rows, channels, width)), dev)
    with _on(dev):
        rc = lib.kda_ssm_conv_bwd_fresh(_ptr(x), xs, dt, _ptr(w), _ptr(bias), _ptr(cache), _ptr(cu_seqlens),
                                        n_seqs, T, channels, width, int(bool(activation)), _ptr(grad_y), gs,
                                        _ptr(gx), _ptr(gw), _ptr(gb), _ptr(gc), _ptr(ws), _nbytes(ws),
                                        _stream(dev), _FRESH_X)
    _status(rc, "kda_ssm_conv_bwd")
    return gx, gw, gb, gc


class _Scan:
    """Checked arguments shared by ssm_chunk_fwd and ssm_chunk_bwd."""

    def __init__(self, x, dt, A, B, C, D, S0, cu_seqlens, dt_bias):
        import torch
        dev, self.dtype = _of(x)
        self.dev = dev
        self.lead, self.n_seqs, self.T = _lead(x, 2, cu_seqlens, "x", dev)
        self.H, self.P = x.shape[-2:]
        if not isinstance(B, torch.Tensor) or B.dim() < 2:
            raise KDAError("B must be [..., G, N]")
        self.G, self.N = B.shape[-2:]
        self.xs = _check_rows(x, "x", self.lead, (self.H, self.P), x.dtype, dev)
        self.bs = _check_rows(B, "B", self.lead, (self.G, self.N), x.dtype, dev)
        self.cs = _check_rows(C, "C", self.lead, (self.G, self.N), x.dtype, dev)
        _check_shape(dt, "dt", self.lead + (self.H,), dev)
        _check_shape(A, "A", (self.H,), dev)
        for name, t in (("D", D), ("dt_bias", dt_bias)):
            if t is not None:
                _check_shape(t, name, (self.H,), dev)
        self.state = (self.n_seqs, self.H, self.N, self.P)
        if S0 is not None:
            _check_shape(S0, "S0", self.state, dev)


def ssm_chunk_fwd_workspace_bytes(n_seqs, T, H, G, N, P, varlen) -> int:
    return int(load_library().kda_ssm_chunk_fwd_workspace_bytes(n_seqs, T, H, G, N, P, int(bool(varlen))))


def ssm_chunk_fwd(x, dt, A, B, C, D=None, S0=None, cu_seqlens=None, *, dt_bias=None, softplus=True,
                  output_final_state=True, y=None, S_T=None, workspace=None, sequence_parallel=True):
    """Selective state space scan of whole sequences (see kda_ssm_chunk_fwd in
    include/kda_ssm.h).

    x [B, T, H, P], B and C [B, T, G, N] (or packed, without the batch axis,
    with cu_seqlens int32 [n_seqs + 1]); dt [B, T, H] float32, before the
    softplus of dt + dt_bias (softplus=False: dt + dt_bias as given); A, D,
    dt_bias [H] float32; S0 [n_seqs, H, N, P] float32 or None.  Returns
    (y like x, contiguous; S_T [n_seqs, H, N, P] float32 or None).
    sequence_parallel=False keeps every sequence on one chain.  Rows of no
    sequence are not written: in a packed batch that has some, a y that is not
    given is undefined there.
    """
    import torch
    lib = load_library()
    a = _Scan(x, dt, A, B, C, D, S0, cu_seqlens, dt_bias)
    if y is None:
        y = _like(x)
    else:
        _check_shape(y, "y", x.shape, a.dev, x.dtype)
    if S_T is not None:
        _check_shape(S_T, "S_T", a.state, a.dev)
    elif output_final_state:
        S_T = torch.empty(a.state, dtype=torch.float32, device=a.dev) if S0 is None else _like(S0)
    ws = None
    if sequence_parallel:
        ws = _workspace(workspace, ssm_chunk_fwd_workspace_bytes(a.n_seqs, a.T, a.H, a.G, a.N, a.P,
                                                                 cu_seqlens is not None), a.dev)
    with _on(a.dev):
        rc = lib.kda_ssm_chunk_fwd(_ptr(x), a.xs, _ptr(B), a.bs, _ptr(C), a.cs, a.dtype, _ptr(dt),
                                   _ptr(dt_bias), int(bool(softplus)), _ptr(A), _ptr(D), _ptr(S0),
                                   _ptr(cu_seqlens), a.n_seqs, a.T, a.H, a.G, a.N, a.P, _ptr(y),
                                   _ptr(S_T), _ptr(ws), _nbytes(ws), _stream(a.dev))
    _status(rc, "kda_ssm_chunk_fwd")
    return y, S_T


def ssm_chunk_bwd_workspace_bytes(dtype, n_seqs, T, H, G, N, P, varlen, groups=None) -> int:
    """Workspace of ssm_chunk_bwd for x of this dtype, with `groups` groups of
    heads at a time (None: all)."""
    import torch
    dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(load_library().kda_ssm_chunk_bwd_workspace_bytes(dt, n_seqs, T, H, G, N, P, int(bool(varlen)),
                                                                G if groups is None else groups))


def ssm_chunk_bwd(x, dt, A, B, C, D, S0, grad_y, grad_S_T=None, cu_seqlens=None, *, dt_bias=None,
                  softplus=True, want_grad_S0=True, grad_x=None, grad_B=None, grad_C=None, workspace=None):
    """Backward pass of ssm_chunk_fwd (see kda_ssm_chunk_bwd in
    include/kda_ssm.h).

    Inputs as for the forward call; grad_y like y; grad_S_T [n_seqs, H, N, P]
    float32 or None.  grad_x, grad_B, grad_C may be given as views of wider
    rows, like x, B and C.  Returns (grad_x, grad_dt, grad_A, grad_B, grad_C,
    grad_D, grad_dt_bias, grad_S0); grad_D and grad_dt_bias are None where D
    and dt_bias are, grad_S0 with want_grad_S0=False.  In packed batches, rows
    of no sequence keep what they held in tensors that are given and are zero
    in the others.
    """
    import torch
    lib = load_library()
    a = _Scan(x, dt, A, B, C, D, S0, cu_seqlens, dt_bias)
    _check_shape(grad_y, "grad_y", x.shape, a.dev, x.dtype)
    if grad_S_T is not None:
        _check_shape(grad_S_T, "grad_S_T", a.state, a.dev)
    outs, fresh = [], _FRESH_DT
    for name, t, like, tail, bit in (("grad_x", grad_x, x, (a.H, a.P), _FRESH_X),
                                     ("grad_B", grad_B, B, (a.G, a.N), _FRESH_B),
                                     ("grad_C", grad_C, C, (a.G, a.N), _FRESH_C)):
        if t is None:
            t = _grad_like(like, a.n_seqs)
            fresh |= bit
        outs.append((t, _check_rows(t, name, a.lead, tail, x.dtype, a.dev)))
    (gx, gxs), (gB, gBs), (gC, gCs) = outs
    gdt, gA = _grad_like(dt, a.n_seqs), _like(A)
    gD = None if D is None else _like(D)
    gbias = None if dt_bias is None else _like(dt_bias)
    like = S0 if S0 is not None else grad_S_T
    gS0 = None if not want_grad_S0 else _like(like) if like is not None else \
        torch.empty(a.state, dtype=torch.float32, device=a.dev)
    ws = _workspace(workspace, ssm_chunk_bwd_workspace_bytes(x.dtype, a.n_seqs, a.T, a.H, a.G, a.N, a.P,
                                                             cu_seqlens is not None), a.dev)
    with _on(a.dev):
        rc = lib.kda_ssm_chunk_bwd_fresh(_ptr(x), a.xs, _ptr(B), a.bs, _ptr(C), a.cs, a.dtype, _ptr(dt),
                                         _ptr(dt_bias), int(bool(softplus)), _ptr(A), _ptr(D), _ptr(S0),
                                         _ptr(cu_seqlens), a.n_seqs, a.T, a.H, a.G, a.N, a.P, _ptr(grad_y),
                                         _ptr(grad_S_T), _ptr(gx), gxs, _ptr(gB), gBs, _ptr(gC), gCs, _ptr(gdt),
                                         _ptr(gA), _ptr(gD), _ptr(gbias), _ptr(gS0), _ptr(ws), _nbytes(ws),
                                         _stream(a.dev), fresh)
    _status(rc, "kda_ssm_chunk_bwd")
    return gx, gdt, gA, gB, gC, gD, gbias, gS0


def ssm_recurrent_fwd(x, dt, A, B, C, S, D=None, *, dt_bias=None, softplus=True, replay=None,
                      n_replay=None, commit=True, y=None):
    """The scan for up to 64 new tokens per request, states in place (see
    kda_ssm_recurrent_fwd in include/kda_ssm.h).

    x [B, T, H, P], dt [B, T, H], B and C [B, T, G, N]; S [B, H, N, P]
    float32.  `replay` = (x, dt, B) of Tr <= 64 tokens per request applied
    first without outputs, n_replay int32 [B] (device) how many of them
    (None: all).  commit=False stores the state right after the replay.
    Returns y [B, T, H, P] in x's dtype.
    """
    import torch
    lib = load_library()
    a = _Scan(x, dt, A, B, C, D, S, None, dt_bias)
    Tr, rx, rdt, rB, rxs, rbs = 0, None, None, None, a.H * a.P, a.G * a.N
    if replay is not None:
        if not isinstance(replay, (tuple, list)) or len(replay) != 3:
            raise KDAError("replay must be (x, dt, B)")
        rx, rdt, rB = replay
        rlead, Br, Tr = _lead(rx, 2, None, "replay x", a.dev)
        if Br != a.n_seqs:
            raise KDAError("replay and x must have the same number of requests")
        rxs = _check_rows(rx, "replay x", rlead, (a.H, a.P), x.dtype, a.dev)
        rbs = _check_rows(rB, "replay B", rlead, (a.G, a.N), x.dtype, a.dev)
        _check_shape(rdt, "replay dt", rlead + (a.H,), a.dev)
    if n_replay is not None:
        _check_shape(n_replay, "n_replay", (a.n_seqs,), a.dev, torch.int32)
    if S is None:
        raise KDAError("S must be a torch.Tensor")
    if y is None:
        y = _like(x)
    else:
        _check_shape(y, "y", x.shape, a.dev, x.dtype)
    with _on(a.dev):
        rc = lib.kda_ssm_recurrent_fwd(_ptr(x), a.xs, _ptr(B), a.bs, _ptr(C), a.cs, a.dtype, _ptr(dt),
                                       _ptr(dt_bias), int(bool(softplus)), _ptr(A), _ptr(D), _ptr(rx),
                                       rxs, _ptr(rB), rbs, _ptr(rdt), _ptr(n_replay), _ptr(S), a.n_seqs,
                                       a.T, Tr, a.H, a.G, a.N, a.P, int(bool(commit)), _ptr(y),
                                       _stream(a.dev))
    _status(rc, "kda_ssm_recurrent_fwd")
    return y


def verify_drafts(p_target, drafts, u, u_next, p_draft=None, n_draft=None, *, workspace=None):
    """Verification of drafted tokens (see kda_verify_drafts in
    include/kda_spec.h).

    p_target [B, K + 1, V] float32 or bfloat16, the target's probabilities
    after each draft; drafts int32 [B, K]; u [B, K] and u_next [B] float32
    uniform numbers; p_draft [B, K, V] the probabilities that the drafts were
    sampled from, or None if they were chosen; n_draft int32 [B] or None.
    Returns (n_accepted int32 [B], tokens int32 [B, K + 1]): the accepted
    drafts, the token that follows them, then -1.
    """
    import torch
    lib = load_library()
    if not isinstance(p_target, torch.Tensor) or p_target.dim() != 3:
        raise KDAError("p_target must be [B, K + 1, V]")
    dev = p_target.device
    _check(p_target, "p_target", None, dev)
    if p_target.dtype not in (torch.bfloat16, torch.float32):
        raise KDAError(f"p_target must be bfloat16 or float32, got {p_target.dtype}")
    dt = _in_dtype(p_target)
    B, K, V = p_target.shape[0], p_target.shape[1] - 1, p_target.shape[2]
    _check_shape(drafts, "drafts", (B, K), dev, torch.int32)
    _check_shape(u, "u", (B, K), dev)
    _check_shape(u_next, "u_next", (B,), dev)
    if p_draft is not None:
        _check_shape(p_draft, "p_draft", (B, K, V), dev, p_target.dtype)
    if n_draft is not None:
        _check_shape(n_draft, "n_draft", (B,), dev, torch.int32)
    n_acc = torch.empty((B,), dtype=torch.int32, device=dev)
    tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    ws = _workspace(workspace, int(lib.kda_verify_drafts_workspace_bytes(B, K, V)), dev)
    with _on(dev):
        rc = lib.kda_verify_drafts(_ptr(p_target), _ptr(p_draft), dt, _ptr(drafts), _ptr(n_draft), _ptr(u),
                                   _ptr(u_next), B, K, V, _ptr(n_acc), _ptr(tokens), _ptr(ws), _nbytes(ws),
                                   _stream(dev))
    _status(rc, "kda_verify_drafts")
    return n_acc, tokens
