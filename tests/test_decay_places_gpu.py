"""Places of the attention's gradients through the wrapper, and a captured backward of a
forward that was not: what the rules on places and streams let pass is right bit by bit."""
import pytest
import torch

from chunkwise_delta_rule_chunk_amd import binding as B
from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

H, G, K, V, T = 4, 2, 64, 32, 300


def _made(seed):
    from chunkwise_delta_rule_chunk_amd import ops
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, do = rn(2, T, H, K), rn(2, T, G, K), rn(2, T, G, V), rn(2, T, H, V)
    g = -torch.rand(H, device="cuda", generator=gen)
    return ops, q, k, v, g, do, ops.decay_attention(q, k, v, g)[2]


def test_gradients_between_each_others_rows():
    ops, q, k, v, g, do, c = _made(1)
    want = ops.decay_attention_backward(c, do)
    # one behind the other in a row, in each order, and with rows of unlike lengths
    for order in ((0, 1, 2), (2, 0, 1), (1, 2, 0)):
        size = (H * K, G * K, G * V)
        row = torch.full((2, T, sum(size) + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        out, at = [None] * 3, 0
        for i in order:
            out[i] = row[..., at:at + size[i]].unflatten(-1, (want[("dq", "dk", "dv")[i]].shape[2], -1))
            at += size[i]
        ops.decay_attention_backward(c, do, out=out)
        assert all(torch.equal(o, want[n]) for o, n in zip(out, ("dq", "dk", "dv"))) and (row[..., -8:] == 7).all()
        late = row[..., 8:8 + size[order[0]]].unflatten(-1, out[order[0]].shape[2:])
        out[order[0]] = late  # eight elements into its neighbour
        with pytest.raises(B.RewyError, match="overlaps"):
            ops.decay_attention_backward(c, do, out=out)
    buf = torch.zeros(2 * T * H * K + 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.RewyError, match="dk overlaps dq"):
        ops.decay_attention_backward(c, do, out=(buf[:2 * T * H * K].view(q.shape), buf[64:64 + 2 * T * G * K].view(k.shape),
                                                 torch.empty_like(v)))
    with pytest.raises(B.RewyError, match="dv overlaps dO"):
        part = do.view(-1)[16:16 + v.numel()].view(v.shape)
        ops.decay_attention_backward(c, do, out=(torch.empty_like(q), torch.empty_like(k), part))


def test_a_captured_backward_of_an_eager_forward():
    ops, q, k, v, g, do, c = _made(2)
    want = ops.decay_attention_backward(c, do)
    n = ops.group_norm(do.flatten(2), groups=H)[3]
    nwant = ops.group_norm_backward(n, do.flatten(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.decay_attention_backward(c, do)
        ngot = ops.group_norm_backward(n, do.flatten(2))
    for _ in range(3):
        for t in (got["dq"], got["dk"], got["dv"], ngot["dx"]):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[x], want[x]) for x in ("dq", "dk", "dv")) and torch.equal(ngot["dx"], nwant["dx"])
        ops.decay_attention(q, k, v, g)  # the program's own work in between
