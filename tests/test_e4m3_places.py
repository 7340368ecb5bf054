"""An output of the e4m3 product that shares bytes with an input is refused, wherever it
begins (no GPU needed)."""
import ctypes

import pytest

from chunkwise_delta_rule_chunk_amd import binding as B

P = ctypes.c_void_p
BASE = 1 << 40
M, N, K = 5, 200, 272
NAMES = ("a", "a_scale", "w", "w_scale", "bias", "y")
BYTES = dict(a=M * K, a_scale=M * 3 * 4, w=N * K, w_scale=2 * 3 * 4, bias=N * 4, y=M * N * 2)


def call(at, as_=0, ys=0):
    d = B.RewyE4m3Desc(M, N, K, 128, 128, B.REWY_BF16, B.REWY_F32, as_, 0, ys)
    return B.rewy_e4m3_linear(d, *(P(at[n]) for n in NAMES), None)


@pytest.mark.parametrize("other", NAMES[:5])
@pytest.mark.parametrize("end", [False, True])
def test_a_shared_byte_is_refused(other, end):
    at = {n: BASE + (i << 30) for i, n in enumerate(NAMES)}
    at["y"] = at[other] + BYTES[other] - 2 if end else at[other] - BYTES["y"] + 2
    assert call(at) == B.REWY_EINVAL and f"y overlaps {other}" in B.rewy_last_error()


def test_rows_between_rows():
    """a and y as parts of one row: apart, unless y is wider than the room that is left (which
    the bias, given at y's last element, shows for the first)."""
    at = {n: BASE + (i << 30) for i, n in enumerate(NAMES)}
    at["y"] = at["a"] + K
    for row, want in ((K + 2 * N, "y overlaps bias"), (K + 2 * N - 16, "y overlaps a")):
        at["bias"] = at["y"] + (M - 1) * row + 2 * N - 4
        assert call(at, row, row // 2) == B.REWY_EINVAL and want in B.rewy_last_error()
