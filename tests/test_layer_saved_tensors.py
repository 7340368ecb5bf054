"""What autograd saves may come back in another layout: hooks that keep saved tensors on
the host or recompute them return contiguous copies.  The backward's descriptor has to
describe the tensors whose addresses it is given with (no GPU: the C calls are stubs that
record their arguments)."""
import contextlib

import pytest
import torch

from chunkwise_delta_rule_chunk_amd import binding as B
from chunkwise_delta_rule_chunk_amd import layer_ops as L


@pytest.fixture
def calls(monkeypatch):
    """The descriptors and addresses of the backward calls, made with CPU tensors."""
    seen = {}

    class On(contextlib.AbstractContextManager):
        def __init__(self, ref, stream, inputs):
            pass

        def __enter__(self):
            return None

        def __exit__(self, *exc):
            return False

    def record(name):
        def call(desc, *args):
            seen[name] = (desc, args)
            return B.REWY_OK
        return call

    monkeypatch.setattr(L, "_On", On)
    for name in ("rewy_ssm_fwd", "rewy_ssm_bwd", "rewy_conv_fwd", "rewy_conv_bwd"):
        monkeypatch.setattr(B, name, record(name))
    return seen


@contextlib.contextmanager
def _copied(kept, change=lambda t: t.clone(memory_format=torch.contiguous_format)):
    def unpack(t):
        t = change(t)
        kept[t.data_ptr()] = t
        return t
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        yield


def _slice(rows, width, first, last, **kw):
    big = torch.randn(1, rows, width, **kw)
    return big[..., first:last].detach().requires_grad_(True)


@pytest.mark.parametrize("cu", [None, [0, 3, 9]])
def test_scan(calls, cu):
    H, V, G, K = 2, 32, 1, 64
    x = _slice(9, 400, 0, H * V).unflatten(-1, (H, V))
    b, c = _slice(9, 400, 64, 64 + K).unflatten(-1, (G, K)), _slice(9, 400, 128, 128 + K).unflatten(-1, (G, K))
    dt, al = torch.zeros(1, 9, H), torch.zeros(H)
    kept = {}
    with _copied(kept):
        y, ht = L.selective_scan_autograd(x, dt, al, b, c, cu_seqlens=cu)
    assert calls["rewy_ssm_fwd"][0].x_stride == 400
    (y.sum() + ht.sum()).backward()
    desc, args = calls["rewy_ssm_bwd"]
    for field, ptr in (("x_stride", args[0]), ("b_stride", args[4]), ("c_stride", args[5])):
        assert getattr(desc, field) == kept[ptr].stride(1), field
    assert (desc.N, bool(desc.cu_seqlens), bool(desc.cu_seqlens_host)) == ((2, True, True) if cu else (0, False, False))


@pytest.mark.parametrize("cu", [None, [0, 3, 9]])
def test_convolution(calls, cu):
    x, w = _slice(9, 50, 3, 23), torch.zeros(20, 4)
    kept = {}
    with _copied(kept):
        y, ht = L.short_conv_autograd(x, w, cu_seqlens=cu)
    assert calls["rewy_conv_fwd"][0].x_stride == 50
    (y.sum() + ht.sum()).backward()
    desc, args = calls["rewy_conv_bwd"]
    assert desc.x_stride == kept[args[0]].stride(1)
    assert (desc.N, bool(desc.cu_seqlens), bool(desc.cu_seqlens_host)) == ((2, True, True) if cu else (0, False, False))


@pytest.mark.parametrize("change,error", [
    (lambda t: t.double(), TypeError),                                   # another type
    (lambda t: t.transpose(-1, -2).contiguous().transpose(-1, -2), ValueError),  # rows not contiguous
])
def test_what_cannot_be_read_is_refused(calls, change, error):
    x, w = _slice(9, 50, 3, 23), torch.zeros(20, 4)
    with _copied({}, change):
        y, _ = L.short_conv_autograd(x, w)
    with pytest.raises(error):
        y.sum().backward()
    args = (torch.randn(1, 9, 2, 32, requires_grad=True), torch.zeros(1, 9, 2), torch.zeros(2), torch.randn(1, 9, 1, 32),
            torch.randn(1, 9, 1, 32))
    with _copied({}, lambda t: change(t) if t.dim() > 1 else t):
        y, _ = L.selective_scan_autograd(*args)
    with pytest.raises(error):
        y.sum().backward()
