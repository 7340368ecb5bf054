"""The norm's 8-bit output is the stored scale's: q = round(y / scale) code by code, the
quotient being the fp32 quotient of what the call returns.

With fp32 rows y is returned as it is formed, so y / scale on the CPU (IEEE division, the
same two operands) has to give every code; nothing is left to a tolerance."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

TOP = {"e4m3": 448.0, "int8": 127.0}


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("M,D,group", [(4000, 1537, 0), (1500, 4096, 128), (20000, 320, 32), (300, 16384, 256)])
def test_codes_are_the_quotients(M, D, group, quant):
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator().manual_seed(M + D)
    x = (torch.randn(M, D, generator=g) * 3).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().float().cuda()
    y, _, q, scale, _ = ops.rms_norm(x, w, quant=quant, group=group)
    y, q, scale = y.cpu(), q.cpu(), scale.cpu()
    n = group or D
    ng = -(-D // n)
    top = torch.nn.functional.pad(y.abs(), (0, ng * n - D)).view(M, ng, n).amax(-1)
    assert torch.equal(scale, top / TOP[quant])
    v = y / scale.repeat_interleave(n, 1)[:, :D]
    if quant == "int8":
        want = torch.round(v).to(torch.int8)
    else:
        want = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    off = (q.view(torch.uint8) != want.view(torch.uint8)).sum().item()
    assert off == 0, f"{off} of {q.numel()} codes are not round(y / scale)"
