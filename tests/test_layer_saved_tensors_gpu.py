"""Autograd with what it saves kept on the host: the gradients of the same call without,
bit by bit, for inputs that are slices of one row (their copies come back contiguous)."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


@pytest.mark.parametrize("packed", [None, "list", "device"])
def test_saved_on_the_host(packed):
    from chunkwise_delta_rule_chunk_amd import ops
    T, H, V, G, K = 150, 2, 32, 1, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    row = rn(1, T, 600).bfloat16().requires_grad_(True)
    cw, nw = rn(H * V + 2 * G * K, 4).requires_grad_(True), rn(H * V).requires_grad_(True)
    dt, al, d = (t.requires_grad_(True) for t in (rn(1, T, H) - 3, rn(H), rn(H)))
    cu = None if packed is None else [0, 70, T]
    if packed == "device":
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    r = rn(1, T, H * V).bfloat16()

    def loss():
        u, ht = ops.short_conv_autograd(row[..., 40:40 + cw.shape[0]], cw, cu_seqlens=cu)
        x, b, c = u.split([H * V, G * K, G * K], -1)
        y, st = ops.selective_scan_autograd(x.unflatten(-1, (H, V)), dt, al, b.unflatten(-1, (G, K)), c.unflatten(-1, (G, K)),
                                            d=d, cu_seqlens=cu)
        z, s = ops.rms_norm_autograd(y.flatten(2), nw, row[..., 300:300 + H * V])
        return (z * r).float().sum() + s.float().sum() + ht.float().sum() + st.sum()

    leaves = (row, cw, nw, dt, al, d)
    want = torch.autograd.grad(loss(), leaves)
    with torch.autograd.graph.save_on_cpu():
        out = loss()
    got = torch.autograd.grad(out, leaves)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_changed_before_the_backward():
    """Offsets that only the GPU holds are part of what the backward reads: overwritten in place
    between the forward and the backward, they are refused as any saved tensor is."""
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(7)
    leaf = lambda *s: torch.randn(*s, generator=g, device="cuda").requires_grad_(True)  # noqa: E731
    x, w = leaf(1, 90, 24), leaf(24, 4)
    args = (leaf(1, 90, 2, 32), leaf(1, 90, 2), leaf(2), leaf(1, 90, 1, 32), leaf(1, 90, 1, 32))
    cu = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")
    for call in (lambda: ops.short_conv_autograd(x, w, cu_seqlens=cu), lambda: ops.selective_scan_autograd(*args, cu_seqlens=cu)):
        y, _ = call()
        cu[1] += 5
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.sum().backward()
        y, _ = call()
        y.sum().backward()
