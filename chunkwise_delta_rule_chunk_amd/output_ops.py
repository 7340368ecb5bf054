"""Torch-facing wrappers of what stands behind a token mixer: the group norm with a
gate or an activation and an 8-bit output, and the product of e4m3 operands that
reads the norms' codes and scales.  They allocate outputs and workspaces with PyTorch
and call the C ABI; no arithmetic happens here.  Streams and workspaces as in
``layer_ops``."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .layer_ops import _DT, _QDT, _QUANT, _adjoint, _check, _dtype, _kept, _like, _like_new, _On, _p, _row_stride, _workspace

_GATE = {None: B.REWY_ACT_NONE, "silu": B.REWY_ACT_SILU, "sigmoid": B.REWY_ACT_SIGMOID}


# ---- group norm -----------------------------------------------------------------
def _norm_problem(x, weight, bias, gate, groups, center, eps, activation, quant, group):
    dt = _dtype(x, "x")
    if activation not in _GATE:
        raise ValueError(f"activation must be None, 'silu' or 'sigmoid' (got {activation!r})")
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'e4m3' or 'int8' (got {quant!r})")
    if group not in (0, 32, 64, 128, 256):
        raise ValueError(f"group must be 0, 32, 64, 128 or 256 (got {group})")
    D = x.shape[-1]
    if not isinstance(groups, int) or groups <= 0 or D % groups:
        raise ValueError(f"groups must divide the {D} channels (got {groups})")
    M = x.numel() // D if D else 0
    wdt = dt
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            wdt = _dtype(t, name)
            _like(t, x, (D,), name)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have one type")
    zs = 0
    if gate is not None:
        if gate.shape != x.shape or gate.dtype != x.dtype:
            raise ValueError("gate must have x's shape and type")
        zs = _row_stride(gate, "gate", 1)
    return B.RewyGnormDesc(M, D, groups, dt, wdt, _GATE[activation], int(bool(center)), _QUANT[quant], group, eps,
                           _row_stride(x, "x", 1), zs, 0, 0, 0)


def group_norm(x, weight=None, bias=None, gate=None, *, groups, center=True, eps=1e-5, activation="silu", quant=None,
               group=0, output=True, stream=None):
    """n = (x - mean) rstd weight + bias over each of ``groups`` runs of neighbouring
    channels of a token (without ``center`` the mean is not taken off), y = n act(gate),
    or act(n) without a gate; ``activation`` "silu", "sigmoid" or None.

    x [..., D] and gate may have a row stride; weight and bias [D].  Returns (y, q, scale,
    ctx): y is None with ``output=False``; with ``quant`` "e4m3" or "int8", q holds y /
    scale in 8 bits with one fp32 scale per row (``group=0``: scale [rows, 1]) or per
    ``group`` columns (scale [rows, ceil(D / group)]; 128 is what ``e4m3_linear``
    reads).  ctx feeds ``group_norm_backward``."""
    desc = _norm_problem(x, weight, bias, gate, groups, center, eps, activation, quant, group)
    M, D = desc.M, desc.D
    with _On(x, stream, (x, weight, bias, gate)) as handle:
        y = _like_new(x) if output else None
        mean = x.new_empty((M, groups), dtype=torch.float32) if center else None
        rstd = x.new_empty((M, groups), dtype=torch.float32)
        q = scale = None
        if quant is not None:
            q = x.new_empty(x.shape, dtype=_QDT[quant])
            scale = x.new_empty((M, -(-D // group) if group else 1), dtype=torch.float32)
        _check(B.rewy_gnorm_fwd(desc, _p(x), _p(gate), _p(weight), _p(bias), _p(y), _p(q), _p(scale), _p(mean),
                                _p(rstd), handle), "rewy_gnorm_fwd")
    return y, q, scale, dict(x=x, weight=weight, bias=bias, gate=gate, mean=mean, rstd=rstd, groups=groups,
                             center=center, eps=eps, activation=activation, stream=handle)


def group_norm_backward(ctx, dy, *, stream=None, ws=None):
    """Gradients of the norm's y: dict(dx, dgate, dweight, dbias).  dy may have a row
    stride."""
    x, weight, bias, gate, mean, rstd = (ctx[k] for k in ("x", "weight", "bias", "gate", "mean", "rstd"))
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    desc = _norm_problem(x, weight, bias, gate, ctx["groups"], ctx["center"], ctx["eps"], ctx["activation"], None, 0)
    desc.y_stride = _row_stride(dy, "dy", 1)
    with _On(x, stream, (x, weight, bias, gate, mean, rstd, dy)) as handle:
        _kept(ctx, handle, x, mean, rstd)
        dx = _like_new(x)
        dz = None if gate is None else _like_new(gate)
        dw = None if weight is None else torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        ws = _workspace(B.rewy_gnorm_workspace_bytes(desc), x, ws)
        _check(B.rewy_gnorm_bwd(desc, _p(x), _p(gate), _p(weight), _p(bias), _p(mean), _p(rstd), _p(dy), _p(dx), _p(dz),
                                _p(dw), _p(db), _p(ws), ws.numel(), handle), "rewy_gnorm_bwd")
    return dict(dx=dx, dgate=dz, dweight=dw, dbias=db)


class GroupNormFunction(torch.autograd.Function):
    """Autograd wrapper: y = GroupNormFunction.apply(x, weight, bias, gate, groups, center, eps, activation)."""

    @staticmethod
    def forward(fctx, x, weight, bias, gate, groups, center, eps, activation):
        y, _, _, ctx = group_norm(x, weight, bias, gate, groups=groups, center=center, eps=eps, activation=activation)
        fctx.save_for_backward(x, weight, bias, gate, ctx["mean"], ctx["rstd"])
        fctx.rest = dict(groups=groups, center=center, eps=eps, activation=activation)
        return y

    @staticmethod
    @once_differentiable
    def backward(fctx, dy):
        x, weight, bias, gate, mean, rstd = fctx.saved_tensors  # (hooks may return them in another layout)
        rows = (x.numel() // x.shape[-1] if x.shape[-1] else 0, fctx.rest["groups"])
        _like(mean, x, rows, "mean", torch.float32)
        _like(rstd, x, rows, "rstd", torch.float32)
        ctx = dict(fctx.rest, x=x, weight=weight, bias=bias, gate=gate, mean=mean, rstd=rstd)
        g = group_norm_backward(ctx, _adjoint(dy, x))
        return g["dx"], g["dweight"], g["dbias"], g["dgate"], None, None, None, None


def group_norm_autograd(x, weight=None, bias=None, gate=None, *, groups, center=True, eps=1e-5, activation="silu"):
    """Differentiable group norm on the HIP path: y."""
    return GroupNormFunction.apply(x, weight, bias, gate, groups, center, eps, activation)


# ---- product of e4m3 operands -----------------------------------------------------
def e4m3_linear(a, a_scale, w, w_scale, bias=None, *, dtype=torch.bfloat16, stream=None):
    """y [..., N] = (a a_scale) (w w_scale)^T + bias for codes a [..., K] and w [N, K] in
    float8_e4m3fn: a and a_scale as the norms hand them out (``quant="e4m3"``; ``group=128``:
    a_scale [rows, ceil(K / 128)], ``group=0``: [rows, 1]), w_scale [ceil(N / 128), ceil(K /
    128)] for blocks of 128 x 128 or [N, ceil(K / 128)] for rows.  ``dtype`` is y's, bf16 or
    fp32.  Rows of a and w may have a stride; K is a multiple of 16.  Sums are fp32 for an fp32
    y and for up to 32 rows; a bf16 y of more rows may also miss 2^-10 of the sum of its terms'
    magnitudes (rewy.h), so a row's bits may depend on how many share the call.  For inference:
    8-bit codes have no gradient."""
    for t, name in ((a, "a"), (w, "w")):
        if t.dtype != torch.float8_e4m3fn:
            raise TypeError(f"{name} must be float8_e4m3fn (got {t.dtype})")
    if w.dim() != 2 or a.dim() < 1 or a.shape[-1] != w.shape[1]:
        raise ValueError("a must be [..., K] and w [N, K]")
    if dtype not in _DT:
        raise TypeError(f"dtype must be bf16 or fp32 (got {dtype})")
    N, K = w.shape
    M = a.numel() // K if K else 0
    if max(M, N, K) >= 1 << 31:
        raise ValueError("a and w have fewer than 2^31 rows")
    nb = -(-K // 128)
    whole = a_scale.dim() == 2 and a_scale.shape[1] == 1 and nb > 1
    _like(a_scale, a, (M, 1 if whole else nb), "a_scale", torch.float32)
    rows = w_scale.dim() == 2 and w_scale.shape[0] == N and N != -(-N // 128)
    _like(w_scale, a, (N if rows else -(-N // 128), nb), "w_scale", torch.float32)
    bdt = B.REWY_F32
    if bias is not None:
        bdt = _dtype(bias, "bias")
        _like(bias, a, (N,), "bias")
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (a, a_scale, w, w_scale, bias)):
        raise ValueError("e4m3_linear has no gradient: detach its inputs or run it under torch.no_grad()")
    desc = B.RewyE4m3Desc(M, N, K, 0 if whole else 128, 1 if rows else 128, _DT[dtype], bdt, _row_stride(a, "a", 1),
                          _row_stride(w, "w", 1), 0)
    with _On(a, stream, (a, a_scale, w, w_scale, bias)) as handle:
        y = a.new_empty((*a.shape[:-1], N), dtype=dtype)
        _check(B.rewy_e4m3_linear(desc, _p(a), _p(a_scale), _p(w), _p(w_scale), _p(bias), _p(y), handle),
               "rewy_e4m3_linear")
    return y
