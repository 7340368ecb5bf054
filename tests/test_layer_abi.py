"""Refusals of the operators around the token mixer, all on the host before
anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

from chunkwise_delta_rule_chunk_amd import binding as B
from chunkwise_delta_rule_chunk_amd import layer_ops as L

P = ctypes.c_void_p
OK = 256  # an aligned address that no call gets as far as using


def _norm(**kw):
    d = dict(M=4, D=100, dtype=B.REWY_BF16, w_dtype=B.REWY_F32, quant=0, group=0, eps=1e-6, x_stride=0, res_stride=0,
             sum_stride=0, y_stride=0)
    d.update(kw)
    return B.RewyNormDesc(*d.values())


@pytest.mark.parametrize("bad,status,msg", [
    (dict(M=-1), B.REWY_EINVAL, "bad shape"), (dict(M=1 << 31), B.REWY_EINVAL, "bad shape"),
    (dict(D=0), B.REWY_EINVAL, "bad shape"), (dict(D=16385), B.REWY_EUNSUPPORTED, "exceeds"),
    (dict(dtype=2), B.REWY_EINVAL, "bad dtype"), (dict(w_dtype=-1), B.REWY_EINVAL, "bad w_dtype"),
    (dict(quant=3), B.REWY_EINVAL, "bad quant"), (dict(group=48), B.REWY_EINVAL, "bad group"),
    (dict(eps=-1.0), B.REWY_EINVAL, "bad eps"), (dict(eps=float("nan")), B.REWY_EINVAL, "bad eps"),
    (dict(x_stride=99), B.REWY_EINVAL, "shorter"), (dict(y_stride=-1), B.REWY_EINVAL, "shorter"),
    (dict(sum_stride=(1 << 31) + 1), B.REWY_EINVAL, "too large"),
])
def test_norm_descriptor(bad, status, msg):
    rc = B.rewy_norm_fwd(_norm(**bad), P(OK), None, None, None, P(OK), None, None, None, None)
    assert rc == status and msg in B.rewy_last_error()
    assert B.rewy_norm_workspace_bytes(_norm(**bad)) == 0


def test_norm_pointers():
    def fwd(d, **kw):
        a = dict(x=OK, res=None, w=None, sum=None, y=OK, q=None, scale=None, rstd=None)
        a.update(kw)
        return B.rewy_norm_fwd(d, *(None if v is None else P(v) for v in a.values()), None)

    for d, kw, msg in ((_norm(), dict(x=None), "x is NULL"), (_norm(), dict(x=OK + 1), "x is not 2-byte"),
                       (_norm(), dict(w=OK + 2), "w is not 4-byte"), (_norm(quant=1), dict(q=OK), "scale is NULL"),
                       (_norm(quant=1), dict(scale=OK), "q is NULL"), (_norm(), dict(q=OK), "only when quant"),
                       (_norm(), dict(scale=OK), "only when quant")):
        assert fwd(d, **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    assert fwd(_norm(M=0), x=None, y=None) == B.REWY_OK  # no rows: nothing to do
    need = B.rewy_norm_workspace_bytes(_norm())
    assert need >= 4 * 100 and need % 256 == 0

    def bwd(d, ws=OK, n=1 << 30, **kw):
        a = dict(s=OK, w=OK, rstd=OK, dy=OK, ds=None, dx=OK, dw=OK)
        a.update(kw)
        return B.rewy_norm_bwd(d, *(None if v is None else P(v) for v in a.values()), None if ws is None else P(ws), n, None)

    for kw, msg in ((dict(s=None), "s is NULL"), (dict(rstd=None), "rstd is NULL"), (dict(dy=None), "dy is NULL"),
                    (dict(dx=None), "dx is NULL"), (dict(w=None), "without w")):
        assert bwd(_norm(), **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    for kw in (dict(n=need - 1), dict(ws=None), dict(ws=OK + 16)):
        assert bwd(_norm(), **kw) == B.REWY_EWORKSPACE
    assert B.load().rewy_norm_fwd(None, *[None] * 9) == B.REWY_EINVAL


def _conv(**kw):
    d = dict(B=2, T=10, D=64, W=4, N=0, cu=None, host=None, dtype=B.REWY_BF16, w_dtype=B.REWY_F32, act=1, x_stride=0,
             y_stride=0, dx_stride=0)
    d.update(kw)
    return B.RewyConvDesc(*d.values())


@pytest.mark.parametrize("bad,status,msg", [
    (dict(B=0), B.REWY_EINVAL, "bad shape"), (dict(T=-1), B.REWY_EINVAL, "bad shape"),
    (dict(B=1 << 16, T=1 << 15), B.REWY_EINVAL, "too large"), (dict(D=0), B.REWY_EINVAL, "bad shape"),
    (dict(W=1), B.REWY_EUNSUPPORTED, "taps"), (dict(W=5), B.REWY_EUNSUPPORTED, "taps"), (dict(W=0), B.REWY_EINVAL, "taps"),
    (dict(N=3), B.REWY_EINVAL, "must equal"), (dict(cu=8), B.REWY_EINVAL, "B == 1"),
    (dict(B=1, cu=8), B.REWY_EINVAL, "N >= 1"), (dict(B=1, cu=9, N=1), B.REWY_EINVAL, "aligned"),
    (dict(dtype=5), B.REWY_EINVAL, "bad dtype"), (dict(w_dtype=5), B.REWY_EINVAL, "bad w_dtype"),
    (dict(act=2), B.REWY_EINVAL, "bad act"), (dict(x_stride=63), B.REWY_EINVAL, "shorter"),
    (dict(dx_stride=1), B.REWY_EINVAL, "shorter"),
])
def test_conv_descriptor(bad, status, msg):
    rc = B.rewy_conv_fwd(_conv(**bad), P(OK), P(OK), None, None, P(OK), None, None)
    assert rc == status and msg in B.rewy_last_error()
    assert B.rewy_conv_workspace_bytes(_conv(**bad)) == 0


def test_conv_pointers():
    for a, msg in (([None, OK, None, None, OK, None], "x is NULL"), ([OK, None, None, None, OK, None], "w is NULL"),
                   ([OK, OK, None, None, None, None], "y is NULL"), ([OK, OK + 2, None, None, OK, None], "w is not 4-byte"),
                   ([OK, OK, None, OK + 1, OK, None], "h0 is not 2-byte")):
        assert B.rewy_conv_fwd(_conv(), *(None if v is None else P(v) for v in a), None) == B.REWY_EINVAL
        assert msg in B.rewy_last_error()
    assert B.rewy_conv_step(_conv(), P(OK), P(OK), None, P(OK), P(OK), P(OK), None) == B.REWY_EINVAL
    assert "T == 1" in B.rewy_last_error()
    assert B.rewy_conv_fwd(_conv(T=0), None, None, None, None, None, None, None) == B.REWY_OK
    cu = (ctypes.c_int32 * 3)(0, 7, 5)
    d = _conv(B=1, N=2, cu=8, host=ctypes.addressof(cu))
    assert B.rewy_conv_workspace_bytes(d) == 0 and "not ascending" in B.rewy_last_error()
    need = B.rewy_conv_workspace_bytes(_conv())

    def bwd(n=need, **kw):
        a = dict(x=OK, w=OK, bias=OK, h0=OK, dy=OK, dht=None, dx=OK, dw=OK, dbias=OK, dh0=OK, ws=OK)
        a.update(kw)
        return B.rewy_conv_bwd(_conv(), *(None if v is None else P(v) for v in a.values()), n, None)

    for kw, msg in ((dict(dbias=None), "exactly when"), (dict(bias=None), "exactly when"), (dict(dh0=None), "dh0 is NULL"),
                    (dict(dw=None), "dw is NULL"), (dict(dx=None), "dx is NULL")):
        assert bwd(**kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    assert bwd(n=need - 1) == B.REWY_EWORKSPACE and bwd(ws=None) == B.REWY_EWORKSPACE


def test_conv_overlaps_and_sizes():
    """Runs read their neighbours' rows, so nothing is formed in place but a step's."""
    A = [P(256 * (i + 1)) for i in range(12)]
    assert B.rewy_conv_fwd(_conv(), A[0], A[1], None, A[2], A[0], None, None) == B.REWY_EINVAL and "y may not" in B.rewy_last_error()
    assert B.rewy_conv_fwd(_conv(), A[0], A[1], None, A[2], A[3], A[2], None) == B.REWY_EINVAL and "ht may not" in B.rewy_last_error()
    need = B.rewy_conv_workspace_bytes(_conv())
    for dx, dh0, msg in ((0, 7, "dx may not"), (4, 7, "dx may not"), (6, 2, "dh0 may not"), (6, 5, "dh0 may not")):
        rc = B.rewy_conv_bwd(_conv(), A[0], A[1], A[3], A[2], A[4], A[5], A[dx], A[8], A[9], A[dh0], A[10], need, None)
        assert rc == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    for kw in (dict(B=1 << 26, T=1, D=1), dict(B=1 << 20, T=1, D=1 << 14), dict(D=(1 << 23) + 1)):
        assert B.rewy_conv_workspace_bytes(_conv(**kw)) == 0, kw
    assert B.rewy_conv_workspace_bytes(_conv(B=1, T=1 << 30, D=1)) > 0


def test_ssm_sizes_and_overlaps():
    """More workgroups than a launch takes are refused, not left to the launch."""
    for kw in (dict(B=1 << 22, T=1, H=8, G=8, K=32, V=32), dict(B=1, T=1 << 30, H=64, G=64, K=32, V=32)):
        for phase in (0, 1):
            assert B.rewy_ssm_workspace_bytes(_ssm(**kw), phase) == 0 and "too many" in B.rewy_last_error()
    assert B.rewy_ssm_workspace_bytes(_ssm(B=1, T=1 << 24, H=32, G=1, K=128, V=64), 0) > 0
    assert B.rewy_ssm_workspace_bytes(_ssm(B=1, T=1 << 20, H=64, G=8, K=128, V=64), 1) > 0
    A = [P(256 * (i + 1)) for i in range(24)]
    need = B.rewy_ssm_workspace_bytes(_ssm(), 1)
    for dh0 in (7, 9):
        # x dt a_log dt_bias b c D h0, dy dht, dx ddt da_log ddt_bias db dc dD dh0
        rc = B.rewy_ssm_bwd(_ssm(), *A[:8], A[8], A[9], *A[10:17], A[dh0], A[20], need, None)
        assert rc == B.REWY_EINVAL and "dh0 may not" in B.rewy_last_error()


def _ssm(**kw):
    d = dict(B=2, T=100, H=4, G=2, K=64, V=32, N=0, cu=None, host=None, dtype=B.REWY_BF16, dt_dtype=B.REWY_F32,
             x_stride=0, b_stride=0, c_stride=0, y_stride=0, dx_stride=0, db_stride=0, dc_stride=0)
    d.update(kw)
    return B.RewySsmDesc(*d.values())


@pytest.mark.parametrize("bad,status,msg", [
    (dict(B=-1), B.REWY_EINVAL, "bad shape"), (dict(H=0), B.REWY_EINVAL, "bad heads"), (dict(G=0), B.REWY_EINVAL, "bad heads"),
    (dict(G=3), B.REWY_EINVAL, "multiple of G"), (dict(K=48), B.REWY_EUNSUPPORTED, "not supported"),
    (dict(V=256), B.REWY_EUNSUPPORTED, "not supported"), (dict(K=0), B.REWY_EINVAL, "bad shape"),
    (dict(dtype=B.REWY_F32, K=128), B.REWY_EUNSUPPORTED, "not supported"), (dict(dtype=9), B.REWY_EINVAL, "bad dtype"),
    (dict(dt_dtype=9), B.REWY_EINVAL, "bad dt_dtype"), (dict(x_stride=120), B.REWY_EINVAL, "shorter"),
    (dict(b_stride=129), B.REWY_EINVAL, "16 bytes"), (dict(c_stride=1 << 23), B.REWY_EUNSUPPORTED, "2^22"),
    (dict(N=1), B.REWY_EINVAL, "must equal"), (dict(cu=8), B.REWY_EINVAL, "B == 1"),
])
def test_ssm_descriptor(bad, status, msg):
    rc = B.rewy_ssm_fwd(_ssm(**bad), *([P(OK)] * 10), P(OK), 1 << 40, None)
    assert rc == status and msg in B.rewy_last_error()
    assert B.rewy_ssm_workspace_bytes(_ssm(**bad), 0) == 0
    assert B.rewy_ssm_workspace_bytes(_ssm(**bad), 1) == 0


def test_ssm_pointers():
    names = ("x", "dt", "a_log", "dt_bias", "b", "c", "D", "h0", "y", "ht")

    def fwd(call=B.rewy_ssm_fwd, ws=OK, n=1 << 40, **kw):
        a = {k: OK for k in names}
        a["ht"] = 4 * OK
        a.update(kw)
        a = [None if v is None else P(v) for v in a.values()]
        tail = [None] if call is B.rewy_ssm_recurrent_fwd else [None if ws is None else P(ws), n, None]
        return call(_ssm(T=3000), *a, *tail)

    for call in (B.rewy_ssm_fwd, B.rewy_ssm_recurrent_fwd):
        for kw, msg in ((dict(x=None), "x is NULL"), (dict(dt=None), "dt is NULL"), (dict(a_log=None), "A_log is NULL"),
                        (dict(b=None), "b is NULL"), (dict(c=None), "c is NULL"), (dict(y=None), "y is NULL"),
                        (dict(x=OK + 8), "x is not 16-byte"), (dict(h0=OK + 4), "h0 is not 16-byte"),
                        (dict(dt=OK + 2), "dt is not 4-byte")):
            assert fwd(call, **kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    assert fwd(ht=OK) == B.REWY_EINVAL and "ht may not be h0" in B.rewy_last_error()
    need = B.rewy_ssm_workspace_bytes(_ssm(T=3000), 0)
    assert need > 0 and fwd(n=need - 1) == B.REWY_EWORKSPACE and fwd(ws=None) == B.REWY_EWORKSPACE
    assert fwd(ws=OK + 128) == B.REWY_EWORKSPACE
    assert B.rewy_ssm_workspace_bytes(_ssm(), 2) == 0 and "bad phase" in B.rewy_last_error()
    need = B.rewy_ssm_workspace_bytes(_ssm(), 1)

    def bwd(n=need, **kw):
        a = {k: OK for k in ("x", "dt", "a_log", "dt_bias", "b", "c", "D", "h0", "dy", "dht", "dx", "ddt", "da_log",
                             "ddt_bias", "db", "dc", "dD", "dh0", "ws")}
        a.update(kw)
        return B.rewy_ssm_bwd(_ssm(), *(None if v is None else P(v) for v in a.values()), n, None)

    for kw, msg in ((dict(dy=None), "dy is NULL"), (dict(dx=None), "dx is NULL"), (dict(ddt=None), "ddt is NULL"),
                    (dict(da_log=None), "dA_log is NULL"), (dict(db=None), "db is NULL"), (dict(dc=None), "dc is NULL"),
                    (dict(dh0=None), "dh0 is NULL"), (dict(dD=None), "dD is NULL"), (dict(D=None), "exactly when"),
                    (dict(dt_bias=None), "exactly when"), (dict(ddt_bias=None), "ddt_bias is NULL")):
        assert bwd(**kw) == B.REWY_EINVAL and msg in B.rewy_last_error(), msg
    assert bwd(n=need - 1) == B.REWY_EWORKSPACE


def test_wrappers_refuse():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        L.rms_norm(x, w)
    with pytest.raises(TypeError, match="bf16 or fp32"):
        L.rms_norm(x.half(), w)
    with pytest.raises(ValueError, match="quant"):
        L.rms_norm(x, w, quant="int4")
    with pytest.raises(ValueError, match="group"):
        L.rms_norm(x, w, quant="int8", group=-1)
    with pytest.raises(ValueError, match="weight must have shape"):
        L.rms_norm(x, torch.zeros(7))
    with pytest.raises(ValueError, match="residual"):
        L.rms_norm(x, w, torch.zeros(2, 7))
    with pytest.raises(ValueError, match="contiguous"):
        L.rms_norm(torch.zeros(8, 2).t(), w)
    x, b, dt, al = torch.zeros(1, 4, 2, 32), torch.zeros(1, 4, 1, 32), torch.zeros(1, 4, 2), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        L.selective_scan(x, dt, al, b, b)
    with pytest.raises(ValueError, match="c must have shape"):
        L.selective_scan(x, dt, al, b, torch.zeros(1, 4, 2, 32))
    with pytest.raises(TypeError, match="b must have x's type"):
        L.selective_scan(x, dt, al, b.bfloat16(), b)
    with pytest.raises(ValueError, match="h0 must have shape"):
        L.selective_scan(x, dt, al, b, b, h0=torch.zeros(2, 2, 32, 32))
    with pytest.raises(TypeError, match="a_log must be"):
        L.selective_scan(x, dt, al.double(), b, b)
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="end at T"):
        L.short_conv(x, torch.zeros(8, 4), cu_seqlens=[0, 3])
    with pytest.raises(ValueError, match="h0 must have shape"):
        L.short_conv(x, torch.zeros(8, 4), h0=torch.zeros(1, 4, 8))
    with pytest.raises(ValueError, match="activation"):
        L.short_conv(x, torch.zeros(8, 4), activation="relu")
    with pytest.raises(ValueError, match="evenly spaced"):
        L.short_conv(torch.zeros(2, 8, 8)[:, :4], torch.zeros(8, 4))
    with pytest.raises(ValueError, match="overlap"):
        L.short_conv(torch.zeros(64).as_strided((1, 4, 8), (32, 2, 1)), torch.zeros(8, 4))
