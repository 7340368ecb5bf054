"""Row counts at the end of 32 bits are refused before anything is enqueued, whatever the
other sizes are (no GPU needed)."""
import ctypes

import pytest

from chunkwise_delta_rule_chunk_amd import binding as B

P = ctypes.c_void_p
MOST = 2 ** 31 - 1024  # rows of a


def _linear(M, N, y=3 * 256):
    d = B.RewyE4m3Desc(M, N, 16, 128, 128, B.REWY_BF16, B.REWY_F32, 0, 0, 0)
    return B.rewy_e4m3_linear(d, P(256), P(256), P(512), P(256), None, None if y is None else P(y), None)


@pytest.mark.parametrize("N", [1, 128, 129, 4000, 1 << 24])
@pytest.mark.parametrize("M", [MOST + 1, 2 ** 31 - 129, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
def test_rows_past_the_limit(M, N):
    assert _linear(M, N, y=None) == B.REWY_EUNSUPPORTED and "too large" in B.rewy_last_error()


def test_rows_up_to_the_limit():
    """One column of tiles: the sizes pass, and the missing pointer is what is refused."""
    for M in (1, 33, MOST):
        assert _linear(M, 128, y=None) == B.REWY_EINVAL and "y is NULL" in B.rewy_last_error()
    assert _linear(MOST, 129, y=None) == B.REWY_EUNSUPPORTED and "too large" in B.rewy_last_error()
