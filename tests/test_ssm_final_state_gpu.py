"""The scan's y is the same bit by bit whether the final state is asked for or not, and with
it everything that tests of the call with a final state show of y."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


@pytest.mark.parametrize("B,T,H,G,K,V,dtype,lens", [
    (1, 1500, 8, 1, 128, 128, "bf16", None),        # several segments
    (2, 1100, 6, 2, 128, 64, "bf16", None),
    (1, 1400, 5, 1, 64, 32, "bf16", [1, 0, 700, 699]),
    (1, 900, 3, 3, 32, 128, "bf16", [300, 600]),
    (1, 200, 4, 1, 128, 128, "bf16", None),         # one
    (1, 700, 4, 2, 64, 64, "fp32", None),
])
def test_y_without_the_final_state(B, T, H, G, K, V, dtype, lens):
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator().manual_seed(T + K + V)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, b, c = (rn(B, T, n, v).to(dt).cuda() for n, v in ((H, V), (G, K), (G, K)))
    step, al, d = (rn(B, T, H) - 4).cuda(), rn(H).cuda(), rn(H).cuda()
    h0 = rn(len(lens) if lens else B, H, K, V).cuda()
    cu = None
    if lens:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
    for kw in (dict(d=d, h0=h0), dict()):
        y, ht, _ = ops.selective_scan(x, step, al, b, c, cu_seqlens=cu, **kw)
        y2, none, _ = ops.selective_scan(x, step, al, b, c, cu_seqlens=cu, output_final_state=False, **kw)
        assert none is None and torch.equal(y, y2)
