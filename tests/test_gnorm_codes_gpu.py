"""The group norm's codes are y divided by the stored scale, rounded once: bit by bit, beside
the borders between codes, for scales of every size down to the smallest.  With x = 1, no
mean, eps = 0 and no activation, n is 1 and y is the gate itself."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

F8 = torch.float8_e4m3fn


def borders(quant):
    """The values halfway between two codes."""
    if quant == "int8":
        return torch.arange(0, 127) + 0.5
    grid = torch.arange(0, 0x7f, dtype=torch.uint8).view(F8).float()
    return (grid[1:] + grid[:-1]) / 2  # (exact)


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("low", [-100, -97, -95, -91, -84, -60, 0, 100, 125])
def test_codes_beside_their_borders(low, quant):
    from chunkwise_delta_rule_chunk_amd import ops
    gen = torch.Generator().manual_seed(200 + low)
    M = 200_000 if low < -80 else 40_000
    top = 448.0 if quant == "e4m3" else 127.0
    amax = torch.exp2(low + 2 * torch.rand(M, 1, generator=gen, dtype=torch.float64)).float()
    scale = amax / top
    t = borders(quant)
    t = t[torch.randint(len(t), (M, 31), generator=gen)]
    v = (scale.double() * t.double()).float()  # the float nearest to the border, or one of its neighbours
    v = (v.view(torch.int32) + torch.randint(-1, 2, v.shape, generator=gen, dtype=torch.int32)).view(torch.float32)
    sign = torch.randint(2, (M, 32), generator=gen) * 2 - 1
    y = torch.cat([amax, torch.minimum(v, amax)], 1) * sign
    for group in (32, 0):
        z = y if group else y[:, :20].contiguous()
        x = torch.ones_like(z).cuda()
        got, q, s, _ = ops.group_norm(x, None, None, z.cuda(), groups=1 if group else 5, center=False, eps=0.0,
                                      activation=None, quant=quant, group=group)
        assert torch.equal(got.cpu(), z) and torch.equal(s.cpu(), scale)
        want = z / scale
        want = want.clamp(-top, top).to(F8).view(torch.uint8) if quant == "e4m3" else want.round().to(torch.int8)
        q = q.cpu().view(want.dtype)
        assert torch.equal(q, want), (q != want).sum()


def test_a_scale_that_is_no_number_keeps_its_codes():
    from chunkwise_delta_rule_chunk_amd import ops
    z = torch.full((3, 32), 2.0, device="cuda")
    z[0, 3], z[1, 4] = float("inf"), float("nan")
    for quant, inf in (("e4m3", None), ("int8", 0)):
        _, q, s, _ = ops.group_norm(torch.ones_like(z), None, None, z, groups=1, center=False, eps=0.0, activation=None,
                                    quant=quant, group=32)
        f = q.float()
        assert torch.isinf(s[0]).all() and torch.isnan(s[1]).all() and s[2] == (torch.tensor(2.0) / (448 if inf is None else 127)).item()
        finite = torch.arange(32, device="cuda") != 3
        assert (f[0][finite] == 0).all()  # a number over infinity
        if quant == "e4m3":
            assert torch.isnan(f[0, 3]) and torch.isnan(f[1]).all() and (f[2] == 448).all()
        else:
            assert f[0, 3] == 0 and (f[1] == 0).all() and (f[2] == 127).all()
