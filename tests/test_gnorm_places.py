"""Outputs of the group norm that share bytes with an input or another output are refused,
wherever they begin (no GPU needed)."""
import ctypes

import pytest

from chunkwise_delta_rule_chunk_amd import binding as B

P = ctypes.c_void_p
BASE = 1 << 40
M, D, G = 5, 96, 3
NAMES = ("x", "z", "w", "b", "y", "q", "scale", "mean", "rstd", "dy", "dx", "dz", "dw", "db", "ws")
ROWS, PAR, STAT = M * D * 2, D * 4, M * G * 4  # bytes


def _far():
    return {n: BASE + (i << 30) for i, n in enumerate(NAMES)}


def _desc(quant, **strides):
    s = [strides.get(n, 0) for n in ("x", "z", "y", "dx", "dz")]
    return B.RewyGnormDesc(M, D, G, B.REWY_BF16, B.REWY_F32, 1, 1, quant, 32 if quant else 0, 1e-5, *s)


def fwd(at, **strides):
    return B.rewy_gnorm_fwd(_desc(1, **strides), *(P(at[n]) for n in NAMES[:9]), None)


def bwd(at, **strides):
    return B.rewy_gnorm_bwd(_desc(0, **strides), *(P(at[n]) for n in ("x", "z", "w", "b", "mean", "rstd", "dy", "dx", "dz", "dw",
                                                                     "db", "ws")), 1 << 40, None)


@pytest.mark.parametrize("call,name,other,off", [
    (fwd, "y", "x", 2), (fwd, "y", "z", -ROWS + 2), (fwd, "y", "w", 4), (fwd, "q", "x", ROWS - 1), (fwd, "q", "y", 0),
    (fwd, "scale", "q", M * D - 4), (fwd, "scale", "b", -M * 3 * 4 + 4), (fwd, "mean", "rstd", STAT - 4), (fwd, "rstd", "scale", 0),
    (fwd, "mean", "x", 0), (fwd, "rstd", "y", ROWS - 4),
    (bwd, "dx", "x", 2), (bwd, "dx", "dy", -2), (bwd, "dz", "z", ROWS - 2), (bwd, "dz", "dx", 2), (bwd, "dw", "w", 4),
    (bwd, "dw", "w", 0), (bwd, "db", "dw", PAR - 4), (bwd, "db", "dw", 0), (bwd, "dw", "rstd", STAT - 4), (bwd, "dx", "mean", 0),
    (bwd, "db", "dy", 0),
])
def test_a_shared_byte_is_refused(call, name, other, off):
    at = _far()
    at[name] = at[other] + off
    assert call(at) == B.REWY_EINVAL
    err = B.rewy_last_error()
    assert "overlaps" in err and name in err and other in err, err


def test_slices_of_one_row():
    """dx and dz as halves of a row of 2 D are apart; one element to the side they are not."""
    for shift, want in ((0, "db overlaps dw"), (2, "dz overlaps dx"), (-2, "dz overlaps dx")):
        at = _far()
        at["dz"] = at["dx"] + D * 2 + shift
        at["db"] = at["dw"] + 4  # (refused for this at the latest)
        assert bwd(at, dx=2 * D, dz=2 * D) == B.REWY_EINVAL and want in B.rewy_last_error()
