"""Refusals of the attention with a constant decay, the group norm and the e4m3 product,
all on the host before anything is enqueued (no GPU needed)."""
import contextlib
import ctypes

import pytest
import torch

from chunkwise_delta_rule_chunk_amd import binding as B
from chunkwise_delta_rule_chunk_amd import decay_ops as DO
from chunkwise_delta_rule_chunk_amd import ops
from chunkwise_delta_rule_chunk_amd import output_ops as OO

P = ctypes.c_void_p
OK = 256  # an aligned address that no call gets as far as using


def _at(v):
    return None if v is None else P(v)


# ---- attention ----------------------------------------------------------------------
def _decay(**kw):
    d = dict(B=2, T=10, H=4, G=2, K=64, V=128, N=0, cu=None, host=None, dtype=B.REWY_BF16, scale=0.1, qs=0, ks=0, vs=0,
             os=0, dqs=0, dks=0, dvs=0)
    d.update(kw)
    return B.RewyDecayDesc(*d.values())


def _decay_fwd(d, ws=OK, n=1 << 40, **kw):
    a = dict(q=OK, k=2 * OK, v=3 * OK, g=OK, h0=None, o=4 * OK, ht=None)
    a.update(kw)
    return B.rewy_decay_fwd(d, *map(_at, a.values()), _at(ws), n, None)


def _decay_bwd(d, ws=OK, n=1 << 40, **kw):
    a = dict(q=OK, k=2 * OK, v=3 * OK, g=OK, h0=None, dO=4 * OK, dht=None, states=None, sn=0, dq=5 * OK, dk=6 * OK,
             dv=7 * OK, dh0=None)
    a.update(kw)
    return B.rewy_decay_bwd(d, *(v if k == "sn" else _at(v) for k, v in a.items()), _at(ws), n, None)


@pytest.mark.parametrize("bad,status,msg", [
    (dict(B=0), B.REWY_EINVAL, "bad shape"), (dict(T=-1), B.REWY_EINVAL, "bad shape"),
    (dict(B=1 << 16, T=1 << 15), B.REWY_EINVAL, "too large"), (dict(N=3), B.REWY_EINVAL, "must equal"),
    (dict(cu=8), B.REWY_EINVAL, "B == 1"), (dict(B=1, cu=8), B.REWY_EINVAL, "N >= 1"),
    (dict(B=1, cu=9, N=1), B.REWY_EINVAL, "aligned"),
    (dict(H=0), B.REWY_EINVAL, "bad heads"), (dict(G=0), B.REWY_EINVAL, "bad heads"), (dict(G=3), B.REWY_EINVAL, "bad heads"),
    (dict(H=2, G=4), B.REWY_EINVAL, "bad heads"), (dict(H=65538), B.REWY_EINVAL, "bad heads"),
    (dict(K=0), B.REWY_EINVAL, "bad shape"), (dict(V=-32), B.REWY_EINVAL, "bad shape"),
    (dict(K=96), B.REWY_EUNSUPPORTED, "not supported"), (dict(V=256), B.REWY_EUNSUPPORTED, "not supported"),
    (dict(dtype=2), B.REWY_EINVAL, "bad dtype"), (dict(scale=float("inf")), B.REWY_EINVAL, "finite"),
    (dict(scale=float("nan")), B.REWY_EINVAL, "finite"), (dict(qs=255), B.REWY_EINVAL, "shorter"),
    (dict(dvs=8), B.REWY_EINVAL, "shorter"), (dict(ks=129), B.REWY_EINVAL, "16 bytes"),
    (dict(vs=(1 << 22) + 8), B.REWY_EUNSUPPORTED, "exceeds"),
    (dict(B=1 << 14, T=1, H=1 << 10, G=1 << 10), B.REWY_EUNSUPPORTED, "too many"),
])
def test_decay_descriptor(bad, status, msg):
    assert _decay_fwd(_decay(**bad)) == status and msg in B.rewy_last_error()
    assert _decay_bwd(_decay(**bad)) == status and msg in B.rewy_last_error()
    assert B.rewy_decay_workspace_bytes(_decay(**bad), 0) == 0
    d = _decay(**bad)
    assert B.rewy_decay_recurrent_fwd(d, *[P(OK)] * 4, None, P(2 * OK), None, None) == status


def test_decay_pointers():
    d = _decay()
    assert B.rewy_decay_workspace_bytes(d, 2) == 0 and B.rewy_decay_workspace_bytes(d, -1) == 0
    for kw, msg in ((dict(q=None), "q is NULL"), (dict(k=None), "k is NULL"), (dict(v=OK + 8), "v is not 16-byte"),
                    (dict(g=None), "g is NULL"), (dict(g=OK + 2), "g is not 4-byte"), (dict(o=None), "o is NULL"),
                    (dict(h0=OK + 4), "h0 is not 16-byte"), (dict(ht=OK + 4), "ht is not 16-byte"),
                    (dict(h0=OK, ht=OK), "ht may not be h0"), (dict(o=OK), "o may not be")):
        assert _decay_fwd(d, **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    for kw, msg in ((dict(dO=None), "dO is NULL"), (dict(dq=None), "dq is NULL"), (dict(dk=None), "dk is NULL"),
                    (dict(dv=OK + 2), "dv is not 16-byte"), (dict(h0=OK), "dh0 is NULL"),
                    (dict(dht=OK + 4), "dht is not 16-byte"), (dict(h0=9 * OK, dh0=9 * OK), "dh0 may not be"),
                    (dict(dht=9 * OK, dh0=9 * OK), "dh0 may not be"), (dict(dq=OK), "may not be an input"),
                    (dict(dv=4 * OK), "may not be an input"), (dict(dk=5 * OK), "places of their own"),
                    (dict(dv=6 * OK), "places of their own")):
        assert _decay_bwd(d, **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    long = _decay(B=1, T=100000, H=4, G=2)
    for phase, call in ((0, _decay_fwd), (1, _decay_bwd)):
        need = B.rewy_decay_workspace_bytes(long, phase)
        assert need % 256 == 0 and need >= 4 * 64 * 128 * 4
        for kw in (dict(n=need - 1), dict(ws=None), dict(ws=OK + 16)):
            assert call(long, **kw) == B.REWY_EWORKSPACE
    need = B.rewy_decay_workspace_bytes(long, 0)
    for kw in (dict(states=OK, sn=need - 1), dict(states=OK + 16, sn=need)):
        assert _decay_bwd(long, **kw) == B.REWY_EWORKSPACE
    # no tokens and no state to hand out: nothing to do
    none = dict(q=None, k=None, v=None)
    assert _decay_fwd(_decay(T=0), o=None, **none) == B.REWY_OK
    assert _decay_bwd(_decay(T=0), dO=None, dq=None, dk=None, dv=None, **none) == B.REWY_OK
    assert B.load().rewy_decay_fwd(None, *[None] * 8, 0, None) == B.REWY_EINVAL


def test_decay_host_offsets():
    def call(*off):
        arr = (ctypes.c_int32 * len(off))(*off)
        return _decay_fwd(_decay(B=1, T=10, N=len(off) - 1, cu=OK, host=ctypes.addressof(arr)), o=None)
    for off in ((1, 10), (0, 5, 4, 10), (0, 11), (0, -1, 10)):
        assert call(*off) == B.REWY_EINVAL and "cu_seqlens" in B.rewy_last_error(), off
    for off in ((0, 4, 4, 10), (0, 9)):  # good offsets: rows may follow the last sequence
        assert call(*off) == B.REWY_EINVAL and "o is NULL" in B.rewy_last_error()


# ---- group norm ----------------------------------------------------------------------
def _gnorm(**kw):
    d = dict(M=4, D=96, G=3, dtype=B.REWY_BF16, w_dtype=B.REWY_F32, act=1, center=1, quant=0, group=0, eps=1e-5, xs=0, zs=0,
             ys=0, dxs=0, dzs=0)
    d.update(kw)
    return B.RewyGnormDesc(*d.values())


def _gnorm_fwd(d, **kw):
    a = dict(x=OK, z=None, w=None, b=None, y=2 * OK, q=None, scale=None, mean=OK, rstd=OK)
    a.update(kw)
    return B.rewy_gnorm_fwd(d, *map(_at, a.values()), None)


def _gnorm_bwd(d, ws=OK, n=1 << 40, **kw):
    a = dict(x=OK, z=None, w=OK, b=None, mean=OK, rstd=OK, dy=2 * OK, dx=3 * OK, dz=None, dw=OK, db=None)
    a.update(kw)
    return B.rewy_gnorm_bwd(d, *map(_at, a.values()), _at(ws), n, None)


@pytest.mark.parametrize("bad,status,msg", [
    (dict(M=-1), B.REWY_EINVAL, "bad shape"), (dict(M=1 << 31), B.REWY_EINVAL, "bad shape"),
    (dict(D=0), B.REWY_EINVAL, "bad shape"), (dict(D=16386), B.REWY_EUNSUPPORTED, "exceeds"),
    (dict(G=0), B.REWY_EINVAL, "divide"), (dict(G=5), B.REWY_EINVAL, "divide"), (dict(G=-3), B.REWY_EINVAL, "divide"),
    (dict(dtype=2), B.REWY_EINVAL, "bad dtype"), (dict(w_dtype=-1), B.REWY_EINVAL, "bad w_dtype"),
    (dict(act=3), B.REWY_EINVAL, "bad act"), (dict(center=2), B.REWY_EINVAL, "bad center"),
    (dict(quant=3), B.REWY_EINVAL, "bad quant"), (dict(group=48), B.REWY_EINVAL, "bad group"),
    (dict(eps=-1.0), B.REWY_EINVAL, "bad eps"), (dict(eps=float("nan")), B.REWY_EINVAL, "bad eps"),
    (dict(xs=95), B.REWY_EINVAL, "shorter"), (dict(zs=-1), B.REWY_EINVAL, "shorter"),
    (dict(ys=(1 << 31) + 1), B.REWY_EINVAL, "too large"), (dict(dzs=5), B.REWY_EINVAL, "shorter"),
])
def test_gnorm_descriptor(bad, status, msg):
    assert _gnorm_fwd(_gnorm(**bad)) == status and msg in B.rewy_last_error()
    assert _gnorm_bwd(_gnorm(**bad)) == status and msg in B.rewy_last_error()
    assert B.rewy_gnorm_workspace_bytes(_gnorm(**bad)) == 0


def test_gnorm_pointers():
    codes = _gnorm(quant=1, group=128)
    for d, kw, msg in ((_gnorm(), dict(x=None), "x is NULL"), (_gnorm(), dict(x=OK + 1), "x is not 2-byte"),
                       (_gnorm(), dict(w=OK + 2), "w is not 4-byte"), (_gnorm(), dict(b=OK + 2), "b is not 4-byte"),
                       (_gnorm(), dict(mean=None), "mean is NULL"), (_gnorm(), dict(rstd=None), "rstd is NULL"),
                       (_gnorm(center=0), dict(), "only with center"), (codes, dict(q=OK), "scale is NULL"),
                       (codes, dict(scale=OK), "q is NULL"), (_gnorm(), dict(q=OK), "only when quant"),
                       (_gnorm(), dict(y=OK), "y may not be"), (_gnorm(), dict(z=2 * OK), "y may not be")):
        assert _gnorm_fwd(d, **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    assert _gnorm_fwd(_gnorm(M=0), x=None, mean=None, rstd=None) == B.REWY_OK
    for kw, msg in ((dict(x=None), "x is NULL"), (dict(dy=None), "dy is NULL"), (dict(dx=None), "dx is NULL"),
                    (dict(rstd=None), "rstd is NULL"), (dict(z=OK), "dz is NULL"), (dict(dz=4 * OK), "only with"),
                    (dict(w=None), "only with"), (dict(db=OK), "only with"), (dict(dx=OK), "may not be an input"),
                    (dict(dx=2 * OK), "may not be an input"), (dict(z=4 * OK, dz=3 * OK), "dx may not be dz")):
        assert _gnorm_bwd(_gnorm(), **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    need = B.rewy_gnorm_workspace_bytes(_gnorm())
    assert need >= 2 * 96 * 4 and need % 256 == 0
    for kw in (dict(n=need - 1), dict(ws=None), dict(ws=OK + 16)):
        assert _gnorm_bwd(_gnorm(), **kw) == B.REWY_EWORKSPACE
    assert B.load().rewy_gnorm_fwd(None, *[None] * 10) == B.REWY_EINVAL


# ---- e4m3 product --------------------------------------------------------------------
def _e4m3(**kw):
    d = dict(M=4, N=100, K=256, a_block=128, w_rows=128, dtype=B.REWY_BF16, bias_dtype=B.REWY_F32, as_=0, ws=0, ys=0)
    d.update(kw)
    return B.RewyE4m3Desc(*d.values())


def _linear(d, **kw):
    a = dict(a=OK, sa=OK, w=2 * OK, sw=OK, bias=None, y=3 * OK)
    a.update(kw)
    return B.rewy_e4m3_linear(d, *map(_at, a.values()), None)


@pytest.mark.parametrize("bad,status,msg", [
    (dict(M=-1), B.REWY_EINVAL, "bad shape"), (dict(N=0), B.REWY_EINVAL, "bad shape"), (dict(K=0), B.REWY_EINVAL, "bad shape"),
    (dict(K=264), B.REWY_EUNSUPPORTED, "multiple of 16"), (dict(K=(1 << 20) + 16), B.REWY_EUNSUPPORTED, "too large"),
    (dict(N=(1 << 24) + 1), B.REWY_EUNSUPPORTED, "too large"), (dict(a_block=64), B.REWY_EINVAL, "bad a_block"),
    (dict(w_rows=64), B.REWY_EINVAL, "bad w_rows"), (dict(dtype=2), B.REWY_EINVAL, "bad dtype"),
    (dict(bias_dtype=2), B.REWY_EINVAL, "bad bias_dtype"), (dict(as_=240), B.REWY_EINVAL, "shorter"),
    (dict(ws=264), B.REWY_EINVAL, "multiples of 16"), (dict(as_=(1 << 22) + 16), B.REWY_EUNSUPPORTED, "exceeds"),
    (dict(ys=99), B.REWY_EINVAL, "shorter"), (dict(M=1 << 24, N=1 << 20), B.REWY_EUNSUPPORTED, "too large"),
])
def test_e4m3_descriptor(bad, status, msg):
    assert _linear(_e4m3(**bad)) == status and msg in B.rewy_last_error()


def test_e4m3_pointers():
    for kw, msg in ((dict(a=None), "a is NULL"), (dict(a=OK + 8), "a is not 16-byte"), (dict(w=None), "w is NULL"),
                    (dict(w=OK + 4), "w is not 16-byte"), (dict(sa=None), "a_scale is NULL"),
                    (dict(sw=OK + 2), "w_scale is not 4-byte"), (dict(bias=OK + 2), "bias is not 4-byte"),
                    (dict(y=None), "y is NULL"), (dict(y=OK + 1), "y is not 2-byte"), (dict(y=OK), "y may not be"),
                    (dict(y=2 * OK), "y may not be")):
        assert _linear(_e4m3(), **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    assert _linear(_e4m3(M=0), a=None, sa=None, w=None, sw=None, y=None) == B.REWY_OK
    assert B.load().rewy_e4m3_linear(None, *[None] * 7) == B.REWY_EINVAL


# ---- wrappers ------------------------------------------------------------------------
def test_wrappers_refuse():
    q, k, v, g = torch.zeros(1, 8, 4, 64), torch.zeros(1, 8, 2, 64), torch.zeros(1, 8, 2, 32), torch.zeros(4)
    for fn in (ops.decay_attention, ops.decay_attention_recurrent, ops.decay_attention_autograd):
        with pytest.raises(ValueError, match="GPU"):
            fn(q, k, v, g)
        with pytest.raises(ValueError, match="must be"):
            fn(q[0], k[0], v[0], g)
        with pytest.raises(TypeError, match="k must have q's type"):
            fn(q, k.bfloat16(), v, g)
        with pytest.raises(TypeError, match="bf16 or fp32"):
            fn(q.half(), k.half(), v.half(), g)
        with pytest.raises(ValueError, match="k must have shape"):
            fn(q, k[..., :32], v, g)
        with pytest.raises(ValueError, match="v must have q's"):
            fn(q, k, v[:, :7], g)
        with pytest.raises(ValueError, match="log_decay must have shape"):
            fn(q, k, v, g[:2])
        with pytest.raises(TypeError, match="log_decay must be"):
            fn(q, k, v, g.double())
        with pytest.raises(ValueError, match="h0 must have shape"):
            fn(q, k, v, g, h0=torch.zeros(2, 4, 64, 32))
        with pytest.raises(ValueError, match="end at T"):
            fn(q, k, v, g, cu_seqlens=[0, 7])
    with pytest.raises(ValueError, match="ht must have shape"):
        ops.decay_attention_recurrent(q, k, v, g, ht=torch.zeros(4, 64, 32))
    with pytest.raises(ValueError, match="overlap"):
        ops.decay_attention(q.as_strided((1, 8, 4, 64), (0, 64, 64, 1)), k, v, g)
    with pytest.raises(ValueError, match="no gradient"):
        ops.decay_attention_autograd(q, k, v, g.clone().requires_grad_(True))

    x = torch.zeros(3, 48)
    with pytest.raises(ValueError, match="GPU"):
        ops.group_norm(x, groups=4)
    for kw, err, msg in ((dict(groups=5), ValueError, "divide"), (dict(groups=0), ValueError, "divide"),
                         (dict(groups=2.0), ValueError, "divide"), (dict(activation="relu"), ValueError, "activation"),
                         (dict(quant="int4"), ValueError, "quant"), (dict(group=48), ValueError, "group"),
                         (dict(weight=torch.zeros(47)), ValueError, "weight must have shape"),
                         (dict(weight=torch.zeros(48), bias=torch.zeros(48).bfloat16()), TypeError, "one type"),
                         (dict(gate=torch.zeros(3, 47)), ValueError, "gate"),
                         (dict(gate=x.bfloat16()), ValueError, "gate"), (dict(gate=torch.zeros(48, 3).t()), ValueError, "contiguous")):
        with pytest.raises(err, match=msg):
            ops.group_norm(x, **dict(dict(groups=4), **kw))

    f8 = torch.float8_e4m3fn
    a, w, sa, sw = torch.zeros(5, 256).to(f8), torch.zeros(200, 256).to(f8), torch.ones(5, 2), torch.ones(2, 2)
    with pytest.raises(ValueError, match="GPU"):
        ops.e4m3_linear(a, sa, w, sw)
    for args, kw, err, msg in (((a.float(), sa, w, sw), {}, TypeError, "a must be float8"),
                               ((a, sa, w.float(), sw), {}, TypeError, "w must be float8"),
                               ((a[:, :128], sa, w, sw), {}, ValueError, "a must be"),
                               ((a, sa[:4], w, sw), {}, ValueError, "a_scale must have shape"),
                               ((a, sa.double(), w, sw), {}, TypeError, "a_scale must be"),
                               ((a, sa, w, sw[:1]), {}, ValueError, "w_scale must have shape"),
                               ((a, sa, w, torch.ones(200, 1)), {}, ValueError, "w_scale must have shape"),
                               ((a, sa, w, sw, torch.zeros(199)), {}, ValueError, "bias must have shape"),
                               ((a, sa, w, sw, torch.zeros(200).half()), {}, TypeError, "bias must be"),
                               ((a, sa, w, sw), dict(dtype=torch.float16), TypeError, "dtype must be"),
                               ((a, sa, w, sw.clone().requires_grad_(True)), {}, ValueError, "no gradient")):
        with pytest.raises(err, match=msg):
            ops.e4m3_linear(*args, **kw)


# ---- what autograd keeps --------------------------------------------------------------
@pytest.fixture
def calls(monkeypatch):
    """The descriptors and addresses of the C calls, made with CPU tensors."""
    seen = {}

    class On(contextlib.nullcontext):
        def __init__(self, *a):
            super().__init__()

    def record(name):
        def call(desc, *args):
            seen[name] = (desc, args)
            return B.REWY_OK
        return call

    for mod in (DO, OO):
        monkeypatch.setattr(mod, "_On", On)
    for name in ("rewy_decay_fwd", "rewy_decay_bwd", "rewy_gnorm_fwd", "rewy_gnorm_bwd"):
        monkeypatch.setattr(B, name, record(name))
    return seen


@contextlib.contextmanager
def _copied(kept):
    def unpack(t):
        t = t.clone(memory_format=torch.contiguous_format)
        kept[t.data_ptr()] = t
        return t
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        yield


@pytest.mark.parametrize("cu", [None, [0, 3, 9]])
def test_backward_describes_what_comes_back(calls, cu):
    """Slices of one row that hooks return as contiguous copies, and the forward's states."""
    row = torch.randn(1, 9, 800).requires_grad_(True)
    q, k, v = row[..., :256].unflatten(-1, (4, 64)), row[..., 256:384].unflatten(-1, (2, 64)), row[..., 400:464].unflatten(-1, (2, 32))
    kept = {}
    with _copied(kept):
        o, ht = ops.decay_attention_autograd(q, k, v, -torch.ones(4), cu_seqlens=cu)
    f = calls["rewy_decay_fwd"][0]
    assert (f.q_stride, f.k_stride, f.v_stride) == (800, 800, 800)
    o.sum().backward()
    d, a = calls["rewy_decay_bwd"]
    assert (d.q_stride, d.k_stride, d.v_stride, d.o_stride) == (256, 128, 64, 128)
    assert all(p in kept for p in (*a[:4], a[7])) and a[8] == kept[a[7]].numel()
    assert a[4] is None and a[12] is None  # no state: no adjoint of it

    z = torch.randn(6, 60)
    x, gate = z[:, :24].detach().requires_grad_(True), z[:, 30:54]
    kept.clear()
    with _copied(kept):
        y = ops.group_norm_autograd(x, torch.ones(24), None, gate, groups=2)
    assert calls["rewy_gnorm_fwd"][0].x_stride == 60
    y.sum().backward()
    d, a = calls["rewy_gnorm_bwd"]
    assert (d.x_stride, d.z_stride) == (24, 24) and all(p in kept for p in (*a[:3], *a[4:6])) and a[3] is None


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("want", [None, True, False])
def test_want_dh0(calls, state, want):
    q = torch.zeros(1, 9, 2, 32)
    _, _, ctx = ops.decay_attention(q, q, q, -torch.ones(2), h0=torch.zeros(1, 2, 32, 32) if state else None)
    g = ops.decay_attention_backward(ctx, q, want_dh0=want)
    assert (g["dh0"] is not None) == (state if want is None else want)
    assert state <= (calls["rewy_decay_bwd"][1][12] is not None)
