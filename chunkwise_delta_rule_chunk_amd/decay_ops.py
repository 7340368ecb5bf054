"""Torch-facing wrappers of the linear attention with one constant decay for each
head: chunked forward and backward, token-serial form, autograd.  They allocate
outputs and workspaces with PyTorch and call the C ABI; no arithmetic happens
here.  Streams and workspaces as in ``layer_ops``."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .layer_ops import (_aligned, _check, _dtype, _kept, _like, _like_new, _On, _p, _row_stride, _saved_problem,
                        _sequences, _workspace)


def _problem(q, k, v, log_decay, h0, scale, cu_seqlens):
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 4:
            raise ValueError("q must be [B, T, H, K], k [B, T, G, K] and v [B, T, G, V]")
        if t.dtype != q.dtype:
            raise TypeError(f"{name} must have q's type")
    Bsz, T, H, K = q.shape
    G, V = v.shape[2:]
    e = _dtype(q, "q")
    if tuple(k.shape) != (Bsz, T, G, K):
        raise ValueError(f"k must have shape {(Bsz, T, G, K)} (got {tuple(k.shape)})")
    if v.shape[:2] != q.shape[:2]:
        raise ValueError("v must have q's batch rows and tokens")
    _like(log_decay, q, (H,), "log_decay", torch.float32)
    n, cu, host = _sequences(q, cu_seqlens, T)
    nseq = n if cu is not None else Bsz
    shape = (nseq, H, K, V)
    _like(h0, q, shape, "h0", torch.float32)
    desc = B.RewyDecayDesc(Bsz, T, H, G, K, V, n, _p(cu), None if host is None else ctypes.addressof(host), e,
                           max(K, 1) ** -0.5 if scale is None else scale, _row_stride(q, "q", 2), _row_stride(k, "k", 2),
                           _row_stride(v, "v", 2), 0, 0, 0, 0)
    return desc, shape, cu, host


def _new_o(q, v, clear=False):
    shape = (*q.shape[:3], v.shape[3])
    return q.new_zeros(shape) if clear else q.new_empty(shape)


def decay_attention(q, k, v, log_decay, *, scale=None, h0=None, cu_seqlens=None, output_final_state=True,
                    clear=False, stream=None, ws=None):
    """o_t = scale S_t^T q_t with S_t = exp(log_decay) S_{t-1} + k_t v_t^T for each head,
    in chunks (prompts, training).

    q [B, T, H, K], k [B, T, G, K], v [B, T, G, V] (slices of longer rows allowed; H / G
    neighbouring heads share a key and value head), log_decay [H] fp32 (at most 0),
    scale (K^-1/2 if None), h0 [N, H, K, V] fp32.  Returns (o, ht or None, ctx); ctx
    feeds ``decay_attention_backward``, with the states of the workspace where it is not the
    caller's own.  A GPU cu_seqlens may end before T: o's rows
    behind the last sequence are then not written, or zeros with ``clear``."""
    desc, shape, cu, host = _problem(q, k, v, log_decay, h0, scale, cu_seqlens)
    with _On(q, stream, (q, k, v, log_decay, h0, cu)) as handle:
        o = _new_o(q, v, clear)
        ht = q.new_empty(shape, dtype=torch.float32) if output_final_state else None
        states, ws = ws is None, _workspace(B.rewy_decay_workspace_bytes(desc, 0), q, ws)
        _check(B.rewy_decay_fwd(desc, _p(q), _p(k), _p(v), _p(log_decay), _p(h0), _p(o), _p(ht), _p(ws),
                                ws.numel(), handle), "rewy_decay_fwd")
    return o, ht, dict(desc=desc, q=q, k=k, v=v, log_decay=log_decay, h0=h0, cu=cu, host=host,
                       states=ws if states else None, stream=handle)


def decay_attention_recurrent(q, k, v, log_decay, *, scale=None, h0=None, cu_seqlens=None, ht=None, stream=None):
    """The same attention token by token (decoding).  Returns (o, ht); ``ht`` may be h0
    itself (updated in place).  o's rows behind the last sequence are not written."""
    desc, shape, cu, host = _problem(q, k, v, log_decay, h0, scale, cu_seqlens)
    _like(ht, q, shape, "ht", torch.float32)
    with _On(q, stream, (q, k, v, log_decay, h0, cu, ht)) as handle:
        o = _new_o(q, v)
        if ht is None:
            ht = q.new_empty(shape, dtype=torch.float32)
        _check(B.rewy_decay_recurrent_fwd(desc, _p(q), _p(k), _p(v), _p(log_decay), _p(h0), _p(o), _p(ht), handle),
               "rewy_decay_recurrent_fwd")
    return o, ht


def decay_attention_backward(ctx, do, dht=None, *, out=None, want_dh0=None, clear=False, stream=None, ws=None):
    """Gradients of the attention: dict(dq, dk, dv, dh0), dk and dv summed over the heads
    that share them.  do [B, T, H, V] may be a slice of longer rows.  ``out=(dq, dk, dv)``
    gives the places of those three (slices of one row, for the joint projection's
    backward; they share no byte with each other or an input); ``clear`` as in the forward, for the gradients that are made here.  dh0 is
    handed out where h0 was given, or as ``want_dh0`` says."""
    q, k, v, log_decay, h0, states = (ctx[n] for n in ("q", "k", "v", "log_decay", "h0", "states"))
    if tuple(do.shape) != (*q.shape[:3], v.shape[3]) or do.dtype != q.dtype:
        raise ValueError("do must have o's shape and type")
    f = ctx["desc"]
    shape = (f.N if ctx["cu"] is not None else f.B, f.H, f.K, f.V)
    _like(dht, q, shape, "dht", torch.float32)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    if out is not None:
        for t, ref, name in zip(out, (q, k, v), ("dq", "dk", "dv")):
            if t.shape != ref.shape or t.dtype != ref.dtype:
                raise ValueError(f"{name} must have the shape and type of its input")
    with _On(q, stream, (q, k, v, log_decay, h0, ctx["cu"], do, dht, states, *(out or ()))) as handle:
        _kept(ctx, handle, q, ctx["cu"], states)
        if out is None:
            out = tuple(_like_new(t, clear) for t in (q, k, v))
        dq, dk, dv = out
        desc = B.RewyDecayDesc(f.B, f.T, f.H, f.G, f.K, f.V, f.N, f.cu_seqlens, f.cu_seqlens_host, f.dtype, f.scale,
                               f.q_stride, f.k_stride, f.v_stride, _row_stride(do, "do", 2),
                               _row_stride(dq, "dq", 2), _row_stride(dk, "dk", 2), _row_stride(dv, "dv", 2))
        # (the entry writes it wherever there is a state)
        dh0 = q.new_empty(shape, dtype=torch.float32) if want_dh0 or h0 is not None else None
        ws = _workspace(B.rewy_decay_workspace_bytes(desc, 1), q, ws)
        _check(B.rewy_decay_bwd(desc, _p(q), _p(k), _p(v), _p(log_decay), _p(h0), _p(do), _p(dht), _p(states),
                                0 if states is None else states.numel(), _p(dq), _p(dk), _p(dv), _p(dh0), _p(ws),
                                ws.numel(), handle), "rewy_decay_bwd")
    return dict(dq=dq, dk=dk, dv=dv, dh0=dh0 if want_dh0 else None)


class DecayAttentionFunction(torch.autograd.Function):
    """Autograd wrapper: o, ht = DecayAttentionFunction.apply(q, k, v, log_decay, h0, scale, cu_seqlens)."""

    @staticmethod
    def forward(fctx, q, k, v, log_decay, h0, scale, cu_seqlens):
        fctx.set_materialize_grads(False)
        fctx.clear = isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda
        o, ht, ctx = decay_attention(q, k, v, log_decay, scale=scale, h0=h0, cu_seqlens=cu_seqlens, clear=fctx.clear)
        fctx.save_for_backward(q, k, v, log_decay, h0, ctx["cu"], ctx["states"])
        fctx.host, fctx.scale = ctx["host"], scale
        return o, ht

    @staticmethod
    @once_differentiable
    def backward(fctx, do, dht):
        names = ("q", "k", "v", "log_decay", "h0")
        *saved, cu, states = fctx.saved_tensors
        desc, _, cu, host = _saved_problem(_problem(*saved, fctx.scale, cu), fctx.host)
        _like(states, saved[0], states.shape, "states", torch.uint8)  # (checked again: _saved_problem)
        ctx = dict(zip(names, saved), desc=desc, cu=cu, host=host, states=states)
        q, v = ctx["q"], ctx["v"]
        do = q.new_zeros((*q.shape[:3], v.shape[3])) if do is None else do
        g = decay_attention_backward(ctx, _aligned(do), _aligned(dht), clear=fctx.clear)
        return g["dq"], g["dk"], g["dv"], None, g["dh0"], None, None


def decay_attention_autograd(q, k, v, log_decay, *, scale=None, h0=None, cu_seqlens=None):
    """Differentiable linear attention with a constant decay for each head on the HIP
    path: (o, ht).  The decay is a constant: one that requires a gradient is refused while
    gradients are recorded."""
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay is a constant of the model and has no gradient (detach it)")
    return DecayAttentionFunction.apply(q, k, v, log_decay, h0, scale, cu_seqlens)
