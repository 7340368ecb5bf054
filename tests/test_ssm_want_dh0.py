"""selective_scan_backward(want_dh0=False): the call works with an initial state and hands out
no adjoint of it (no GPU: the C call is a stub that makes the library's own checks)."""
import contextlib

import pytest
import torch

from chunkwise_delta_rule_chunk_amd import binding as B
from chunkwise_delta_rule_chunk_amd import layer_ops as L


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("want", [None, True, False])
def test_want_dh0(monkeypatch, state, want):
    seen = {}

    def bwd(desc, *args):
        seen.update(h0=args[7], dh0=args[17])
        # what the entry requires: an adjoint's place wherever there is a state
        return B.REWY_EINVAL if args[7] is not None and args[17] is None else B.REWY_OK

    class On(contextlib.nullcontext):
        def __init__(self, *a):
            super().__init__()

    monkeypatch.setattr(L, "_On", On)
    monkeypatch.setattr(B, "rewy_ssm_fwd", lambda *a: B.REWY_OK)
    monkeypatch.setattr(B, "rewy_ssm_bwd", bwd)
    x, b = torch.zeros(1, 9, 2, 32), torch.zeros(1, 9, 1, 32)
    _, _, ctx = L.selective_scan(x, torch.zeros(1, 9, 2), torch.zeros(2), b, b,
                                 h0=torch.zeros(1, 2, 32, 32) if state else None)
    g = L.selective_scan_backward(ctx, x, want_dh0=want)
    assert (g["dh0"] is not None) == (state if want is None else want)
    assert (seen["h0"] is not None) == state
