"""Torch-facing wrappers of the operators around the token mixer: RMS norm with
the residual's addition and an 8-bit output, short causal convolution,
selective state space scan.  Like
the wrappers of the delta rule they allocate outputs and workspaces with
PyTorch and call the C ABI; no arithmetic happens here.

Streams: work goes to ``stream`` (default: the device's current stream).  On
another stream than the current one, outputs and workspaces are allocated on it
and the inputs are marked as used by it; the caller orders the two streams as
for any torch operation."""
from __future__ import annotations

import contextlib
import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import binding as B

_DT = {torch.bfloat16: B.REWY_BF16, torch.float32: B.REWY_F32}
_QUANT = {None: B.REWY_QUANT_NONE, "e4m3": B.REWY_QUANT_E4M3, "int8": B.REWY_QUANT_INT8}
_QDT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_ACT = {None: B.REWY_ACT_NONE, "silu": B.REWY_ACT_SILU}


def _p(t):
    return None if t is None else t.data_ptr()


def _check(rc, where):
    if rc != B.REWY_OK:
        raise B.RewyError(rc, where)


def _dtype(t, what):
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be bf16 or fp32 (got {t.dtype})")
    return dt


def _like(t, ref, shape, what, dtype=None):
    """A given tensor is on ref's device, with this shape and type, and contiguous."""
    if t is None:
        return
    if t.get_device() != ref.get_device():
        raise ValueError(f"{what} is on {t.device}, not on {ref.device}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _row_stride(t, what, inner):
    """Elements between the rows of t, whose last ``inner`` dimensions are one
    row: a row's elements are contiguous and the rows are evenly spaced."""
    if t.is_contiguous():
        n = 1
        for k in t.shape[len(t.shape) - inner:]:
            n *= k
        return n
    shape, stride = t.shape, t.stride()
    need = 1
    for i in range(len(shape) - 1, len(shape) - 1 - inner, -1):
        if shape[i] != 1 and stride[i] != need:
            raise ValueError(f"{what}: the elements of a row must be contiguous")
        need *= shape[i]
    rows = [(shape[i], stride[i]) for i in range(len(shape) - 1 - inner, -1, -1) if shape[i] != 1]
    if not rows:
        return need
    out = rows[0][1]
    for (n, st), (_, nxt) in zip(rows, rows[1:]):
        if nxt != n * st:
            raise ValueError(f"{what}: rows must be evenly spaced")
    if out < need:
        raise ValueError(f"{what}: rows must not overlap")
    return out


class _On:
    """Device and stream of one call: allocations inside belong to the stream."""
    __slots__ = ("handle", "stack")

    def __init__(self, ref, stream, inputs):
        if not ref.is_cuda:
            raise ValueError(f"tensors must be on a GPU (got {ref.device})")
        idx = ref.get_device()
        for t in inputs:
            if t is not None and t.get_device() != idx:
                raise ValueError(f"all tensors must be on {ref.device} (got one on {t.device})")
        self.stack = None
        if stream is None and torch._C._cuda_getDevice() == idx:  # the usual call, kept short
            self.handle = torch._C._cuda_getCurrentRawStream(idx)
            return
        cur = torch.cuda.current_stream(idx)
        if stream is None:
            stream = cur
        elif stream.device != ref.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {ref.device}")
        self.handle = stream.cuda_stream
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(ref.device))
        self.stack.enter_context(torch.cuda.stream(stream))
        if stream != cur:
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


def _kept(ctx, handle, ref, *tensors):
    """What the forward made for its backward belongs to the forward's stream, and the caller may
    not know of it: on another stream (the call's is the current one here) it is marked as used."""
    if ctx.get("stream", handle) != handle:
        stream = torch.cuda.current_stream(ref.device)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _workspace(nbytes, ref, ws):
    if nbytes == 0:  # (the call itself would refuse the descriptor)
        raise B.RewyError(B.REWY_EINVAL, "workspace size")
    if ws is None:
        return ref.new_empty(nbytes, dtype=torch.uint8)
    if ws.dtype != torch.uint8 or ws.get_device() != ref.get_device() or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {ref.device}")
    ws.record_stream(torch.cuda.current_stream(ref.device))  # (the call's)
    return ws


def _like_new(ref, clear=False):
    """A new contiguous tensor of ref's shape and type on its device; ``clear``: of
    zeros.  (Autograd clears where rows may follow the last sequence, with offsets
    that only the GPU holds: their gradients go on into other products.)"""
    if clear:
        return ref.new_zeros(ref.shape)
    return torch.empty_like(ref) if ref.is_contiguous() else ref.new_empty(ref.shape)


def _adjoint(dy, ref):
    """The adjoint of an output of ref's shape, zeros if nothing used the output."""
    return ref.new_zeros(ref.shape) if dy is None else dy.contiguous()


def _aligned(t):
    """t, contiguous, at a multiple of 16 bytes: autograd may send back a view at any
    offset of a larger buffer."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


# ---- RMS norm -----------------------------------------------------------------
def rms_norm(x, weight=None, residual=None, *, eps=1e-6, quant=None, group=0, output=True,
             stream=None):
    """y = s (mean(s^2) + eps)^-1/2 weight over the last dimension, s = x + residual.

    Returns (y, s, q, scale, ctx): s is the stored sum (x itself without a
    residual); y is None with ``output=False``; with ``quant`` "e4m3" or "int8",
    q holds y / scale in 8 bits with one fp32 scale per row (``group=0``: scale
    [rows, 1]) or per ``group`` columns (scale [rows, ceil(D / group)]).  x and
    residual may have a row stride.  ctx feeds ``rms_norm_backward``."""
    dt = _dtype(x, "x")
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'e4m3' or 'int8' (got {quant!r})")
    if group not in (0, 32, 64, 128, 256):
        raise ValueError(f"group must be 0, 32, 64, 128 or 256 (got {group})")
    D = x.shape[-1]
    M = x.numel() // D if D else 0
    wdt = dt
    if weight is not None:
        wdt = _dtype(weight, "weight")
        _like(weight, x, (D,), "weight")
    xs = _row_stride(x, "x", 1)
    rs = 0
    if residual is not None:
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("residual must have x's shape and type")
        rs = _row_stride(residual, "residual", 1)
    with _On(x, stream, (x, weight, residual)) as handle:
        s = _like_new(x) if residual is not None else None
        y = _like_new(x) if output else None
        rstd = x.new_empty(M, dtype=torch.float32)
        q = scale = None
        if quant is not None:
            q = x.new_empty(x.shape, dtype=_QDT[quant])
            scale = x.new_empty((M, -(-D // group) if group else 1), dtype=torch.float32)
        desc = B.RewyNormDesc(M, D, dt, wdt, _QUANT[quant], group, eps, xs, rs, 0, 0)
        _check(B.rewy_norm_fwd(desc, _p(x), _p(residual), _p(weight), _p(s), _p(y), _p(q), _p(scale),
                               _p(rstd), handle), "rewy_norm_fwd")
    if s is None:
        s = x
    return y, s, q, scale, dict(s=s, weight=weight, rstd=rstd, eps=eps, stream=handle)


def rms_norm_backward(ctx, dy, ds=None, *, stream=None, ws=None):
    """Gradients of the norm's y (and, through ``ds``, of the stored sum).
    Returns dict(dx, dweight); dx is the gradient of x and of the residual."""
    s, weight = ctx["s"], ctx["weight"]
    D = s.shape[-1]
    M = s.numel() // D if D else 0
    for t, name in ((dy, "dy"), (ds, "ds")):
        if t is not None and (t.shape != s.shape or t.dtype != s.dtype):
            raise ValueError(f"{name} must have x's shape and type")
    wdt = _DT[s.dtype] if weight is None else _DT[weight.dtype]
    desc = B.RewyNormDesc(M, D, _DT[s.dtype], wdt, B.REWY_QUANT_NONE, 0, ctx["eps"],
                          _row_stride(s, "s", 1), 0 if ds is None else _row_stride(ds, "ds", 1), 0,
                          _row_stride(dy, "dy", 1))
    with _On(s, stream, (s, weight, ctx["rstd"], dy, ds)) as handle:
        _kept(ctx, handle, s, ctx["rstd"])
        dx = _like_new(s)
        dw = None if weight is None else torch.empty_like(weight)
        if dw is not None:
            ws = _workspace(B.rewy_norm_workspace_bytes(desc), s, ws)
        _check(B.rewy_norm_bwd(desc, _p(s), _p(weight), _p(ctx["rstd"]), _p(dy), _p(ds), _p(dx),
                               _p(dw), _p(ws), 0 if ws is None else ws.numel(), handle),
               "rewy_norm_bwd")
    return dict(dx=dx, dweight=dw)


class RMSNormFunction(torch.autograd.Function):
    """Autograd wrapper: y, s = RMSNormFunction.apply(x, weight, residual, eps)."""

    @staticmethod
    def forward(fctx, x, weight, residual, eps):
        fctx.set_materialize_grads(False)
        y, s, _, _, ctx = rms_norm(x, weight, residual, eps=eps)
        fctx.save_for_backward(s, weight, ctx["rstd"])
        fctx.eps, fctx.residual = eps, residual is not None
        return y, (s if residual is not None else x.view_as(x))

    @staticmethod
    @once_differentiable
    def backward(fctx, dy, ds):
        s, weight, rstd = fctx.saved_tensors  # (checked again: _saved_problem)
        _like(weight, s, s.shape[-1:], "weight")
        _like(rstd, s, (s.shape[:-1].numel(),), "rstd", torch.float32)
        g = rms_norm_backward(dict(s=s, weight=weight, rstd=rstd, eps=fctx.eps), _adjoint(dy, s),
                              None if ds is None else ds.contiguous())
        return g["dx"], g["dweight"], g["dx"] if fctx.residual else None, None


def rms_norm_autograd(x, weight=None, residual=None, *, eps=1e-6):
    """Differentiable RMS norm on the HIP path: (y, s) with s = x + residual."""
    return RMSNormFunction.apply(x, weight, residual, eps)


# ---- sequences ------------------------------------------------------------------
def _sequences(x, cu_seqlens, T):
    """(N for the descriptor, device cu_seqlens or None, host copy or None).  A
    GPU tensor (int32) is used as it is and not looked at by the host; a list
    or host tensor is checked and copied."""
    if cu_seqlens is None:
        return 0, None, None
    if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
            raise TypeError("a GPU cu_seqlens must be a vector of int32")
        _like(cu_seqlens, x, cu_seqlens.shape, "cu_seqlens")
        return cu_seqlens.numel() - 1, cu_seqlens, None
    vals = [int(v) for v in (cu_seqlens.tolist() if hasattr(cu_seqlens, "tolist") else cu_seqlens)]
    if len(vals) < 2:
        raise ValueError("cu_seqlens needs at least two offsets")
    if vals[-1] != T:
        raise ValueError(f"cu_seqlens must end at T={T}")
    host = (ctypes.c_int32 * len(vals))(*vals)
    return len(vals) - 1, torch.tensor(vals, dtype=torch.int32, device=x.device), host


def _saved_problem(problem, host):
    """The problem of tensors that autograd saved, with the forward's host copy of the
    offsets.  Hooks on saved tensors may return them in another layout (contiguous, from
    the host), so strides, types and shapes are those of what came back, not the forward's."""
    desc, shape, cu, own = problem
    if host is not None:
        desc.cu_seqlens_host, own = ctypes.addressof(host), host
    return desc, shape, cu, own


# ---- short convolution ------------------------------------------------------------
def _conv_problem(x, weight, bias, h0, activation, cu_seqlens, step=False):
    if x.dim() != (2 if step else 3):
        raise ValueError("x must be [N, D]" if step else "x must be [B, T, D]")
    if activation not in _ACT:
        raise ValueError(f"activation must be None or 'silu' (got {activation!r})")
    Bsz, T, D = (x.shape[0], 1, x.shape[1]) if step else x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    dt, wdt = _dtype(x, "x"), _dtype(weight, "weight")
    _like(weight, x, (D, W), "weight")
    _like(bias, x, (D,), "bias", weight.dtype)
    n, cu, host = _sequences(x, cu_seqlens, T)
    nseq = n if cu is not None else Bsz
    _like(h0, x, (nseq, W - 1, D), "h0", x.dtype)
    desc = B.RewyConvDesc(Bsz, T, D, W, n, _p(cu), None if host is None else ctypes.addressof(host),
                          dt, wdt, _ACT[activation], _row_stride(x, "x", 1), 0, 0)
    return desc, (nseq, W - 1, D), cu, host


def short_conv(x, weight, bias=None, *, activation="silu", h0=None, cu_seqlens=None,
               output_final_state=False, clear=False, stream=None):
    """Causal convolution of x [B, T, D] with weight [D, W] (W = 2 .. 4) along the
    tokens, bias [D] and SiLU (``activation=None``: none).  h0 [N, W-1, D] holds
    the rows before each sequence (oldest first).  Returns (y, ht or None,
    ctx); ht is the next call's h0, ctx feeds ``short_conv_backward``.  x may be
    a slice of longer rows.  A GPU cu_seqlens may end before T: y's rows behind
    the last sequence are then not written, or zeros with ``clear``."""
    desc, hshape, cu, host = _conv_problem(x, weight, bias, h0, activation, cu_seqlens)
    with _On(x, stream, (x, weight, bias, h0, cu)) as handle:
        y = _like_new(x, clear)
        ht = x.new_empty(hshape) if output_final_state else None
        _check(B.rewy_conv_fwd(desc, _p(x), _p(weight), _p(bias), _p(h0), _p(y), _p(ht), handle),
               "rewy_conv_fwd")
    return y, ht, dict(desc=desc, x=x, weight=weight, bias=bias, h0=h0, cu=cu, host=host, stream=handle)


def short_conv_step(x, h0, weight, bias=None, *, activation="silu", ht=None, stream=None):
    """One new token x [N, D] for each sequence with state h0 [N, W-1, D].
    Returns (y, ht); ``ht`` may be h0 itself (updated in place)."""
    desc, hshape, _, _ = _conv_problem(x, weight, bias, h0, activation, None, step=True)
    _like(ht, x, hshape, "ht", x.dtype)
    if h0 is None:
        raise ValueError("h0 must be given")
    with _On(x, stream, (x, weight, bias, h0, ht)) as handle:
        y = _like_new(x)
        if ht is None:
            ht = x.new_empty(hshape)
        _check(B.rewy_conv_step(desc, _p(x), _p(weight), _p(bias), _p(h0), _p(y), _p(ht), handle),
               "rewy_conv_step")
    return y, ht


def short_conv_backward(ctx, dy, dht=None, *, clear=False, stream=None, ws=None):
    """Gradients of the convolution: dict(dx, dweight, dbias, dh0).  dy [B, T, D]
    may have a token stride; dht [N, W-1, D] is the final state's adjoint; ``clear``
    as in the forward, for dx."""
    x, weight, bias, h0 = (ctx[k] for k in ("x", "weight", "bias", "h0"))
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    d = ctx["desc"]
    hshape = (d.N if ctx["cu"] is not None else d.B, d.W - 1, d.D)
    _like(dht, x, hshape, "dht", x.dtype)
    desc = B.RewyConvDesc(d.B, d.T, d.D, d.W, d.N, d.cu_seqlens, d.cu_seqlens_host, d.dtype, d.w_dtype,
                          d.act, d.x_stride, _row_stride(dy, "dy", 1), 0)
    with _On(x, stream, (x, weight, bias, h0, ctx["cu"], dy, dht)) as handle:
        _kept(ctx, handle, x, ctx["cu"])
        dx = _like_new(x, clear)
        dw = torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        dh0 = None if h0 is None else torch.empty_like(h0)
        ws = _workspace(B.rewy_conv_workspace_bytes(desc), x, ws)
        _check(B.rewy_conv_bwd(desc, _p(x), _p(weight), _p(bias), _p(h0), _p(dy), _p(dht), _p(dx),
                               _p(dw), _p(db), _p(dh0), _p(ws), ws.numel(), handle), "rewy_conv_bwd")
    return dict(dx=dx, dweight=dw, dbias=db, dh0=dh0)


class ShortConvFunction(torch.autograd.Function):
    """Autograd wrapper: y, ht = ShortConvFunction.apply(x, weight, bias, h0, activation, cu_seqlens)."""

    @staticmethod
    def forward(fctx, x, weight, bias, h0, activation, cu_seqlens):
        fctx.set_materialize_grads(False)
        fctx.clear = isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda
        y, ht, ctx = short_conv(x, weight, bias, activation=activation, h0=h0, cu_seqlens=cu_seqlens,
                                output_final_state=True, clear=fctx.clear)
        fctx.save_for_backward(x, weight, bias, h0, ctx["cu"])
        fctx.activation, fctx.host = activation, ctx["host"]
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(fctx, dy, dht):
        x, weight, bias, h0, cu = fctx.saved_tensors
        desc, _, cu, host = _saved_problem(_conv_problem(x, weight, bias, h0, fctx.activation, cu), fctx.host)
        ctx = dict(desc=desc, x=x, weight=weight, bias=bias, h0=h0, cu=cu, host=host)
        g = short_conv_backward(ctx, _adjoint(dy, ctx["x"]), None if dht is None else dht.contiguous(),
                                clear=fctx.clear)
        return g["dx"], g["dweight"], g["dbias"], g["dh0"], None, None


def short_conv_autograd(x, weight, bias=None, *, activation="silu", h0=None, cu_seqlens=None):
    """Differentiable short convolution on the HIP path: (y, ht)."""
    return ShortConvFunction.apply(x, weight, bias, h0, activation, cu_seqlens)


# ---- selective state space scan ---------------------------------------------------
def _scan_problem(x, dt, a_log, b, c, d, dt_bias, h0, cu_seqlens):
    if x.dim() != 4 or b.dim() != 4:
        raise ValueError("x must be [B, T, H, V], b and c [B, T, G, K]")
    Bsz, T, H, V = x.shape
    G, K = b.shape[2:]
    e = _dtype(x, "x")
    for t, name in ((b, "b"), (c, "c")):
        if t.dtype != x.dtype:
            raise TypeError(f"{name} must have x's type")
        if tuple(t.shape) != (Bsz, T, G, K):
            raise ValueError(f"{name} must have shape {(Bsz, T, G, K)} (got {tuple(t.shape)})")
    dte = _dtype(dt, "dt")
    _like(dt, x, (Bsz, T, H), "dt")
    for t, name in ((a_log, "a_log"), (d, "d"), (dt_bias, "dt_bias")):
        _like(t, x, (H,), name, torch.float32)
    n, cu, host = _sequences(x, cu_seqlens, T)
    nseq = n if cu is not None else Bsz
    shape = (nseq, H, K, V)
    _like(h0, x, shape, "h0", torch.float32)
    desc = B.RewySsmDesc(Bsz, T, H, G, K, V, n, _p(cu), None if host is None else ctypes.addressof(host),
                         e, dte, _row_stride(x, "x", 2), _row_stride(b, "b", 2), _row_stride(c, "c", 2),
                         0, 0, 0, 0)
    return desc, shape, cu, host


def selective_scan(x, dt, a_log, b, c, *, d=None, dt_bias=None, h0=None, cu_seqlens=None,
                   output_final_state=True, clear=False, stream=None, ws=None):
    """y_t = S_t^T C_t + d x_t with S_t = exp(-exp(a_log) dt_t) S_{t-1} + dt_t B_t x_t^T
    and dt_t = softplus(dt + dt_bias), in chunks (prompts, training).

    x [B, T, H, V], b and c [B, T, G, K] (slices of longer rows allowed), dt [B, T, H]
    (before the softplus), a_log, d, dt_bias [H] fp32, h0 [N, H, K, V] fp32.
    Returns (y, ht or None, ctx); ctx feeds ``selective_scan_backward``.  A GPU
    cu_seqlens may end before T: y's rows behind the last sequence are then not
    written, or zeros with ``clear``."""
    desc, shape, cu, host = _scan_problem(x, dt, a_log, b, c, d, dt_bias, h0, cu_seqlens)
    with _On(x, stream, (x, dt, a_log, b, c, d, dt_bias, h0, cu)) as handle:
        y = _like_new(x, clear)
        ht = x.new_empty(shape, dtype=torch.float32) if output_final_state else None
        ws = _workspace(B.rewy_ssm_workspace_bytes(desc, 0), x, ws)
        _check(B.rewy_ssm_fwd(desc, _p(x), _p(dt), _p(a_log), _p(dt_bias), _p(b), _p(c), _p(d), _p(h0),
                              _p(y), _p(ht), _p(ws), ws.numel(), handle), "rewy_ssm_fwd")
    return y, ht, dict(desc=desc, x=x, dt=dt, a_log=a_log, b=b, c=c, d=d, dt_bias=dt_bias, h0=h0, cu=cu,
                       host=host, stream=handle)


def selective_scan_recurrent(x, dt, a_log, b, c, *, d=None, dt_bias=None, h0=None, cu_seqlens=None, ht=None,
                             stream=None):
    """The same scan token by token (decoding).  Returns (y, ht); ``ht`` may be
    h0 itself (updated in place)."""
    desc, shape, cu, host = _scan_problem(x, dt, a_log, b, c, d, dt_bias, h0, cu_seqlens)
    _like(ht, x, shape, "ht", torch.float32)
    with _On(x, stream, (x, dt, a_log, b, c, d, dt_bias, h0, cu, ht)) as handle:
        y = _like_new(x)
        if ht is None:
            ht = x.new_empty(shape, dtype=torch.float32)
        _check(B.rewy_ssm_recurrent_fwd(desc, _p(x), _p(dt), _p(a_log), _p(dt_bias), _p(b), _p(c), _p(d),
                                        _p(h0), _p(y), _p(ht), handle), "rewy_ssm_recurrent_fwd")
    return y, ht


def selective_scan_backward(ctx, dy, dht=None, *, out=None, want_dh0=None, clear=False, stream=None, ws=None):
    """Gradients of the scan: dict(dx, ddt, da_log, db, dc, dd, ddt_bias, dh0).
    dy may be a slice of longer rows.  ``out=(dx, db, dc)`` gives the places of
    those three (slices of one row, for the convolution's backward); ``clear`` as in
    the forward, for the gradients that are made here.  dh0 is handed out where h0 was
    given, or as ``want_dh0`` says."""
    x, dt, a_log, b, c, d, dt_bias, h0 = (ctx[k] for k in ("x", "dt", "a_log", "b", "c", "d", "dt_bias",
                                                           "h0"))
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    f = ctx["desc"]
    shape = (f.N if ctx["cu"] is not None else f.B, f.H, f.K, f.V)
    _like(dht, x, shape, "dht", torch.float32)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    if out is not None:
        for t, ref, name in zip(out, (x, b, c), ("dx", "db", "dc")):
            if t.shape != ref.shape or t.dtype != ref.dtype:
                raise ValueError(f"{name} must have the shape and type of its input")
    with _On(x, stream, (x, dt, a_log, b, c, d, dt_bias, h0, ctx["cu"], dy, dht, *(out or ()))) as handle:
        _kept(ctx, handle, x, ctx["cu"])
        if out is None:
            out = tuple(_like_new(t, clear) for t in (x, b, c))
        dx, db, dc = out
        desc = B.RewySsmDesc(f.B, f.T, f.H, f.G, f.K, f.V, f.N, f.cu_seqlens, f.cu_seqlens_host, f.dtype,
                             f.dt_dtype, f.x_stride, f.b_stride, f.c_stride, _row_stride(dy, "dy", 2),
                             _row_stride(dx, "dx", 2), _row_stride(db, "db", 2), _row_stride(dc, "dc", 2))
        ddt, da_log = _like_new(dt, clear), torch.empty_like(a_log)
        dd = None if d is None else torch.empty_like(d)
        ddt_bias = None if dt_bias is None else torch.empty_like(dt_bias)
        # (the entry writes it wherever there is a state)
        dh0 = x.new_empty(shape, dtype=torch.float32) if want_dh0 or h0 is not None else None
        ws = _workspace(B.rewy_ssm_workspace_bytes(desc, 1), x, ws)
        _check(B.rewy_ssm_bwd(desc, _p(x), _p(dt), _p(a_log), _p(dt_bias), _p(b), _p(c), _p(d), _p(h0),
                              _p(dy), _p(dht), _p(dx), _p(ddt), _p(da_log), _p(ddt_bias), _p(db), _p(dc),
                              _p(dd), _p(dh0), _p(ws), ws.numel(), handle), "rewy_ssm_bwd")
    return dict(dx=dx, ddt=ddt, da_log=da_log, db=db, dc=dc, dd=dd, ddt_bias=ddt_bias,
                dh0=dh0 if want_dh0 else None)


class SelectiveScanFunction(torch.autograd.Function):
    """Autograd wrapper: y, ht = SelectiveScanFunction.apply(x, dt, a_log, b, c, d, dt_bias, h0, cu_seqlens)."""

    @staticmethod
    def forward(fctx, x, dt, a_log, b, c, d, dt_bias, h0, cu_seqlens):
        fctx.set_materialize_grads(False)
        fctx.clear = isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda
        y, ht, ctx = selective_scan(x, dt, a_log, b, c, d=d, dt_bias=dt_bias, h0=h0, cu_seqlens=cu_seqlens,
                                    clear=fctx.clear)
        fctx.save_for_backward(x, dt, a_log, b, c, d, dt_bias, h0, ctx["cu"])
        fctx.host = ctx["host"]
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(fctx, dy, dht):
        names = ("x", "dt", "a_log", "b", "c", "d", "dt_bias", "h0")
        saved = fctx.saved_tensors
        desc, _, cu, host = _saved_problem(_scan_problem(*saved), fctx.host)
        ctx = dict(zip(names, saved), desc=desc, cu=cu, host=host)
        g = selective_scan_backward(ctx, _aligned(_adjoint(dy, ctx["x"])), _aligned(dht), clear=fctx.clear)
        return (g["dx"], g["ddt"], g["da_log"], g["db"], g["dc"], g["dd"], g["ddt_bias"], g["dh0"], None)


def selective_scan_autograd(x, dt, a_log, b, c, *, d=None, dt_bias=None, h0=None, cu_seqlens=None):
    """Differentiable selective state space scan on the HIP path: (y, ht)."""
    return SelectiveScanFunction.apply(x, dt, a_log, b, c, d, dt_bias, h0, cu_seqlens)
