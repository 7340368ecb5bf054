"""Adjoints as other operations send them back: contiguous views at any offset (a
concatenation's), expanded ones (a sum's), slices.  Bit by bit the gradients of the same
values in a tensor of their own."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def _grads(outs, wrap, leaves, seed=1):
    """Gradients of the leaves when the outputs, through ``wrap``, meet fixed values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    loss = 0
    for o in outs:
        r = torch.randn(o.shape, generator=g, device="cuda").to(o.dtype)
        loss = loss + wrap(o, r)
    return torch.autograd.grad(loss.sum(), leaves)


def _plain(o, r):
    return (o * r).float().sum()


def _behind(n):
    """The output behind n other values: its adjoint is a view n elements into a buffer."""
    def wrap(o, r):
        z = torch.zeros(n, dtype=o.dtype, device=o.device)
        return (torch.cat([z, o.flatten()]) * torch.cat([z, r.flatten()])).float().sum()
    return wrap


def _padded(o, r):
    """The output as a slice of longer rows: its adjoint is strided."""
    pad = lambda t: torch.nn.functional.pad(t, (1, 2))  # noqa: E731
    return (pad(o) * pad(r)).float().sum()


WRAPS = {"behind 1": _behind(1), "behind 3": _behind(3), "behind 8": _behind(8), "padded": _padded}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", list(WRAPS))
def test_scan(how, dtype):
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(3)
    leaf = lambda *s, d=dtype: torch.randn(*s, generator=g, device="cuda").to(d).requires_grad_(True)  # noqa: E731
    f = torch.float32
    args = (leaf(2, 70, 2, 32), leaf(2, 70, 2), leaf(2, d=f), leaf(2, 70, 1, 32), leaf(2, 70, 1, 32))
    kw = dict(d=leaf(2, d=f), dt_bias=leaf(2, d=f), h0=leaf(2, 2, 32, 32, d=f))
    leaves = (*args, *kw.values())
    want = _grads(ops.selective_scan_autograd(*args, **kw), _plain, leaves)
    got = _grads(ops.selective_scan_autograd(*args, **kw), WRAPS[how], leaves)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", list(WRAPS))
def test_convolution_and_norm(how, dtype):
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(4)
    leaf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype).requires_grad_(True)  # noqa: E731
    x, w, b, h0 = leaf(2, 40, 36), leaf(36, 4), leaf(36), leaf(2, 3, 36)
    run = lambda: ops.short_conv_autograd(x, w, b, h0=h0)  # noqa: E731
    assert all(torch.equal(p, q) for p, q in zip(_grads(run(), _plain, (x, w, b, h0)), _grads(run(), WRAPS[how], (x, w, b, h0))))
    r, nw = leaf(2, 40, 36), leaf(36)
    run = lambda: ops.rms_norm_autograd(x, nw, r)  # noqa: E731
    assert all(torch.equal(p, q) for p, q in zip(_grads(run(), _plain, (x, nw, r)), _grads(run(), WRAPS[how], (x, nw, r))))


def test_expanded():
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(5)
    leaf = lambda *s: torch.randn(*s, generator=g, device="cuda").requires_grad_(True)  # noqa: E731
    args = (leaf(1, 70, 2, 32), leaf(1, 70, 2), leaf(2), leaf(1, 70, 1, 32), leaf(1, 70, 1, 32))
    a = torch.autograd.grad(ops.selective_scan_autograd(*args)[0].sum(), args)
    y = ops.selective_scan_autograd(*args)[0]
    b = torch.autograd.grad(y, args, torch.ones_like(y))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
