"""Sequences longer than a segment may be, with heads enough to fill the chip by themselves:
against the token-serial form in 32 bits for some of the heads (a state takes three roundings
a token there, at most four and a half a chunk here; magnitudes from the same form on
absolute values)."""
import pytest
import torch

from layer_util import DT, U32, close
from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


@pytest.mark.parametrize("dtype,H", [("bf16", 512), ("fp32", 512)])
def test_more_tokens_than_a_segment(dtype, H):
    from chunkwise_delta_rule_chunk_amd import ops
    gen = torch.Generator(device="cuda").manual_seed(9)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(DT[dtype])  # noqa: E731
    T, K, V = 32768 + 300, 32, 32
    q, k, v, do = rn(1, T, H, K), rn(1, T, 1, K), rn(1, T, 1, V), rn(1, T, H, V)
    g = -torch.logspace(-6, 0, H, device="cuda")
    h0, dht = rn(1, H, K, V).float(), rn(1, H, K, V).float()
    o, ht, c = ops.decay_attention(q, k, v, g, h0=h0)
    dq, dh0 = (ops.decay_attention_backward(c, do, dht)[n] for n in ("dq", "dh0"))
    some = torch.tensor([0, 100, H - 1], device="cuda")
    qs, gs, hs = q[:, :, some].contiguous(), g[some], h0[:, some].contiguous()
    s, st = ops.decay_attention_recurrent(qs.float(), k.float(), v.float(), gs, h0=hs)
    m, mt = ops.decay_attention_recurrent(qs.float().abs(), k.float().abs(), v.float().abs(), gs, h0=hs.abs())
    fp = 1.01 * (600 + 4 * T + T / 16) * U32
    op = 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -16 if dtype == "bf16" else 0
    close(o[:, :, some], s, (fp + op) * m, "o")
    close(ht[:, some], st, fp * mt, "ht")
    # the gradients of these heads by themselves, in many segments
    _, _, c = ops.decay_attention(qs, k, v, gs, h0=hs)
    r = ops.decay_attention_backward(c, do[:, :, some].contiguous(), dht[:, some].contiguous())
    bound = 4 * 2.0 ** -8 if dtype == "bf16" else 2e-5
    assert (dq[:, :, some].double() - r["dq"].double()).norm() <= bound * r["dq"].double().norm()
    assert (dh0[:, some].double() - r["dh0"].double()).norm() <= 2e-5 * r["dh0"].double().norm()
