"""The norm's sum over x or the residual, and its gradient over ds, need the same row stride: with
another one a row would overwrite one that is still to be read.  Refused on the host (no GPU)."""
import ctypes

from chunkwise_delta_rule_chunk_amd import binding as B

P = ctypes.c_void_p


def _desc(M=4, D=100, xs=0, rs=0, ss=0, ys=0):
    return B.RewyNormDesc(M, D, B.REWY_BF16, B.REWY_F32, 0, 0, 1e-6, xs, rs, ss, ys)


def _fwd(d, sum_is):
    a = dict(x=P(256), res=P(512), w=None, sum=P(256 if sum_is == "x" else 512), y=P(1024))
    return B.rewy_norm_fwd(d, *a.values(), None, None, P(2048), None)


def test_sum_over_an_input():
    for d, over in ((_desc(xs=200), "x"), (_desc(ss=200), "x"), (_desc(rs=300, ss=200), "res"), (_desc(xs=200), "x")):
        assert _fwd(d, over) == B.REWY_EINVAL and "same stride" in B.rewy_last_error()


def test_gradient_over_ds():
    for d in (_desc(rs=200), _desc(ss=200), _desc(rs=300, ss=200)):
        rc = B.rewy_norm_bwd(d, P(256), None, P(512), P(1024), P(2048), P(2048), None, None, 0, None)
        assert rc == B.REWY_EINVAL and "same stride" in B.rewy_last_error()


def test_gradient_over_other_inputs():
    """dx over s or dy is not among the overlaps that are allowed."""
    for k, name in ((256, "s"), (1024, "dy")):
        rc = B.rewy_norm_bwd(_desc(ss=200), P(256), None, P(512), P(1024), None, P(k), None, None, 0, None)
        assert rc == B.REWY_EINVAL and "same stride" in B.rewy_last_error(), name
