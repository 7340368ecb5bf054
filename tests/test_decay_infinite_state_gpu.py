"""An infinite element of the attention's initial state: in the recurrence it stays what it
is (each decay here is at least 2^-100 over the whole sequence) and makes the outputs of its
column infinite with the query's sign; everything else is as with a zero in its place."""
import pytest
import torch

from layer_util import DT
from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,K,V", [(1, 64, 64), (30, 32, 128), (64, 64, 32), (130, 64, 64), (700, 128, 128), (1000, 32, 32)])
def test_an_infinite_state(T, K, V, dtype):
    from chunkwise_delta_rule_chunk_amd import ops
    gen = torch.Generator(device="cuda").manual_seed(T + K)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    H = 4
    q, k, v = (rn(2, T, h, d).to(DT[dtype]) for h, d in ((H, K), (2, K), (2, V)))
    # (a power of two, whose low part is zero, the others with parts of both signs)
    g = torch.tensor([0.0, -1e-3, -0.0123, -0.069], device="cuda")
    h0 = rn(2, H, K, V)
    at = [(n, h, (7 * h + 3 * n) % K, (5 * h + n) % V, (1.0, -1.0)[(n + h) % 2]) for n in range(2) for h in range(H)]
    zero, inf = h0.clone(), h0.clone()
    for n, h, i, j, sign in at:
        zero[n, h, i, j], inf[n, h, i, j] = 0.0, sign * float("inf")
    for fn in (ops.decay_attention, ops.decay_attention_recurrent):
        o0, ht0 = fn(q, k, v, g, h0=zero)[:2]
        o, ht = fn(q, k, v, g, h0=inf)[:2]
        for n, h, i, j, sign in at:
            assert ht[n, h, i, j] == inf[n, h, i, j], (fn.__name__, n, h, ht[n, h, i, j])
            assert torch.equal(o[n, :, h, j].float(), torch.sign(q[n, :, h, i].float()) * sign * float("inf")), (fn.__name__, n, h)
            ht[n, h, i, j], o[n, :, h, j] = ht0[n, h, i, j], o0[n, :, h, j]
        assert torch.equal(o, o0) and torch.equal(ht, ht0)
