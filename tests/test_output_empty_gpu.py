"""The attention with a constant decay, the group norm and the e4m3 product on calls without
rows or tokens and on single rows given as vectors."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

F8 = torch.float8_e4m3fn


def test_a_norm_without_rows():
    from chunkwise_delta_rule_chunk_amd import ops
    for shape in ((0, 48), (3, 0, 48)):
        x = torch.randn(*shape, device="cuda").requires_grad_()
        w, b = (torch.randn(48, device="cuda").requires_grad_() for _ in range(2))
        y, q, s, _ = ops.group_norm(x.detach(), w.detach(), b.detach(), groups=4, quant="e4m3", group=32)
        assert y.shape == q.shape == x.shape and s.shape == (0, 2)
        ops.group_norm_autograd(x, w, b, groups=4).sum().backward()
        assert x.grad.shape == x.shape and not w.grad.any() and not b.grad.any()  # (sums of nothing)


def test_a_product_without_rows_and_of_a_vector():
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator().manual_seed(1)
    w, sw, bias = torch.randn(70, 144, generator=g).to(F8).cuda(), torch.rand(1, 2, generator=g).cuda(), torch.randn(70, generator=g).cuda()
    assert ops.e4m3_linear(w[:0], torch.empty(0, 2, device="cuda"), w, sw, bias).shape == (0, 70)
    a, sa = torch.randn(1, 144, generator=g).to(F8).cuda(), torch.rand(1, 2, generator=g).cuda()
    y = ops.e4m3_linear(a[0], sa, w, sw, bias, dtype=torch.float32)
    assert y.shape == (70,) and torch.equal(y, ops.e4m3_linear(a, sa, w, sw, bias, dtype=torch.float32)[0])


@pytest.mark.parametrize("packed", [False, True])
def test_an_attention_without_tokens(packed):
    """The state passes through, forward and backward."""
    from chunkwise_delta_rule_chunk_amd import ops
    n, H, K, V = 3, 2, 64, 32
    b, cu = (1, torch.zeros(n + 1, dtype=torch.int32, device="cuda")) if packed else (n, None)
    q, k, v = (torch.empty(b, 0, H, d, device="cuda", dtype=torch.bfloat16).requires_grad_() for d in (K, K, V))
    h0 = torch.randn(n, H, K, V, device="cuda").requires_grad_()
    g = -torch.ones(H, device="cuda")
    o, ht = ops.decay_attention_autograd(q, k, v, g, h0=h0, cu_seqlens=cu)
    assert o.shape == (b, 0, H, V) and torch.equal(ht, h0)
    r = torch.randn_like(ht)
    (ht * r).sum().backward()
    assert torch.equal(h0.grad, r) and q.grad.shape == q.shape
    o, ht = ops.decay_attention_recurrent(q.detach(), k.detach(), v.detach(), g, h0=h0.detach(), cu_seqlens=cu)
    assert torch.equal(ht, h0)
    _, none, c = ops.decay_attention(q.detach(), k.detach(), v.detach(), g, cu_seqlens=cu, output_final_state=False)
    assert none is None and ops.decay_attention_backward(c, o)["dh0"] is None
