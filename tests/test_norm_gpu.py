"""RMS norm with the residual's addition and the 8-bit outputs, against the
formula in 64 bits.

Bounds.  With fp32 arithmetic (half a step U = 2^-24), s = x + res carries U |s|;
the sum of squares of a row is at most 16 terms in a lane and 10 joining steps, all
positive, so rstd is within about 20 U of itself (the root halves it, division and
root add 2 U); y takes three more products: 40 U |y| covers them.  Outputs add
half a step of their type."""
import pytest
import torch

from layer_util import DT, U32, close
from parity_util import gpu_available, say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

EPS = 1e-6


def _inputs(M, D, dtype, wdt, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, D, generator=g)
    x[:, seed % D] *= 15
    r = torch.randn(M, D, generator=g) * 2 if residual else None
    w = 1 + 0.2 * torch.randn(D, generator=g)
    c = lambda t, d: None if t is None else t.to(d).cuda()  # noqa: E731
    return c(x, DT[dtype]), c(r, DT[dtype]), c(w, DT[wdt])


def _formula(x, r, w):
    s = x.double() + (0 if r is None else r.double())
    rstd = (s.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return s, rstd, s * rstd * (1 if w is None else w.double())


SHAPES = [(1, 1), (3, 5), (257, 63), (5, 64), (7, 65), (33, 128), (4, 500), (9, 1000), (3, 1537), (6, 2048),
          (5, 4096), (3, 5000), (2, 8192), (2, 16383), (2, 16384), (70000, 8)]


@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("M,D", SHAPES)
def test_forward_and_backward(M, D, dtype, wdt):
    from chunkwise_delta_rule_chunk_amd import ops
    residual = (M + D) % 3 != 0
    x, r, w = _inputs(M, D, dtype, wdt, M + D, residual)
    s64, rstd, y64 = _formula(x, r, w)
    y, s, _, _, ctx = ops.rms_norm(x, w, r, eps=EPS)
    close(y, y64, 40 * U32 * y64.abs(), "y")
    if residual:
        close(s, s64, U32 * s64.abs(), "s")
    else:
        assert s is x
    close(ctx["rstd"], rstd[:, 0], 25 * U32 * rstd[:, 0], "rstd")

    g = torch.Generator().manual_seed(7)
    dy = torch.randn(M, D, generator=g).to(DT[dtype]).cuda()
    ds = torch.randn(M, D, generator=g).to(DT[dtype]).cuda() if residual else None
    gr = ops.rms_norm_backward(ctx, dy, ds)
    row, k = s.double(), ctx["rstd"].double()[:, None]  # the backward's own inputs
    u = dy.double() * w.double()
    c = (u * row).mean(-1, keepdim=True) * k * k
    dx = k * (u - row * c) + (0 if ds is None else ds.double())
    # c sums terms of both signs: its error goes by their magnitudes
    mag = k * (u.abs() + row.abs() * (u * row).abs().mean(-1, keepdim=True) * k * k)
    close(gr["dx"], dx, 40 * U32 * (mag + (0 if ds is None else ds.double().abs())), "dx")
    terms = dy.double() * row * k
    # at most M / 1024 + 1 rows in a register, then 16 + 64 joining steps
    close(gr["dweight"], terms.sum(0), (M / 1024 + 100) * U32 * terms.abs().sum(0), "dweight")


def test_backward_is_the_forwards_derivative():
    """dx and dw against central differences of the formula in 64 bits."""
    from chunkwise_delta_rule_chunk_amd import ops
    x, r, w = _inputs(3, 37, "fp32", "fp32", 5)
    dy = torch.randn(3, 37, generator=torch.Generator().manual_seed(1)).cuda()
    y, s, _, _, ctx = ops.rms_norm(x, w, r, eps=EPS)
    gr = ops.rms_norm_backward(ctx, dy)

    def loss(xd, wd):
        return (_formula(xd, r, wd)[2] * dy.double()).sum()

    h = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 36)):
        e = torch.zeros(3, 37, dtype=torch.float64, device="cuda")
        e[i, j] = h
        num = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * h)
        assert abs(num.item() - gr["dx"][i, j].item()) < 1e-5 * max(1, abs(num.item()))
        e = torch.zeros(37, dtype=torch.float64, device="cuda")
        e[j] = h
        num = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * h)
        assert abs(num.item() - gr["dweight"][j].item()) < 1e-5 * max(1, abs(num.item()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("quant,group", [("e4m3", 0), ("e4m3", 128), ("e4m3", 32), ("int8", 0), ("int8", 64),
                                         ("int8", 256)])
@pytest.mark.parametrize("M,D", [(1, 3), (5, 33), (9, 100), (4, 128), (3, 1537), (7, 4096), (2, 16384)])
def test_eight_bit_outputs(M, D, quant, group, dtype):
    from chunkwise_delta_rule_chunk_amd import ops
    x, r, w = _inputs(M, D, dtype, "fp32", 3 * M + D)
    _, _, y64 = _formula(x, r, w)
    y, _, q, scale, _ = ops.rms_norm(x, w, r, eps=EPS, quant=quant, group=group, output=False)
    assert y is None and q.shape == x.shape
    g = group or D
    ng = -(-D // g)
    pad = torch.nn.functional.pad(y64, (0, ng * g - D)).view(M, ng, g)
    top = 448.0 if quant == "e4m3" else 127.0
    ref = pad.abs().amax(-1) / top
    close(scale, ref, 45 * U32 * ref, "scale")
    full = scale.double().repeat_interleave(g, 1)[:, :D]
    v = y64 / full
    # half a step of the 8-bit type at the value, and the value's own fp32 error
    half = (torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) if quant == "e4m3"
            else torch.full_like(v, 0.5))
    off = ((q.double() - v).abs() / (half + 60 * U32 * v.abs())).max().item()
    say(f"[layer] q {quant} group {group}: worst error {off:.3f} of half a step")
    assert off <= 1.0
    assert q.double().abs().max() == top  # the largest value takes the largest code


def test_rows_that_hold_nothing_or_are_not_finite():
    from chunkwise_delta_rule_chunk_amd import ops
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(3)).cuda()
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    x[4] = 1e-40  # below the smallest normal number: the mean square is 0
    for quant in ("e4m3", "int8"):
        y, _, q, scale, _ = ops.rms_norm(x, None, None, eps=EPS, quant=quant)
        assert torch.isfinite(y[[0, 1, 4, 5]]).all() and (y[1] == 0).all()
        assert torch.isnan(y[2]).all() and not torch.isfinite(scale[2]).any() and not torch.isfinite(scale[3]).any()
        assert scale[1] == 1 and (q[1].float() == 0).all() and scale[4] == 1 and (q[4].float() == 0).all()
        alone = ops.rms_norm(x[5:].contiguous(), None, None, eps=EPS, quant=quant)
        assert torch.equal(y[5:], alone[0]) and torch.equal(q[5:].view(torch.uint8), alone[2].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_alignment_and_no_rows(dtype):
    """Rows inside longer rows, at every alignment, give the contiguous rows' results bit by bit."""
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator().manual_seed(11)
    big = torch.randn(9, 1300, generator=g).to(DT[dtype]).cuda()
    w = torch.randn(701, generator=g).cuda()
    for off in (0, 1, 3):
        x, r = big[:, off:off + 701], big[:, 580 + off:580 + off + 701]
        a = ops.rms_norm(x, w, r, quant="int8", group=64)
        b = ops.rms_norm(x.contiguous(), w, r.contiguous(), quant="int8", group=64)
        for u, v in zip(a[:4], b[:4]):
            assert torch.equal(u, v)
        dy = big[:, 7 + off:708 + off]
        ga, gb = ops.rms_norm_backward(a[4], dy, x), ops.rms_norm_backward(b[4], dy.contiguous(), x.contiguous())
        assert torch.equal(ga["dx"], gb["dx"]) and torch.equal(ga["dweight"], gb["dweight"])
    e = big[:0, :701]
    y, s, q, scale, ctx = ops.rms_norm(e, w, e, quant="e4m3")
    assert y.shape == (0, 701) and scale.shape == (0, 1)
    assert (ops.rms_norm_backward(ctx, e)["dweight"] == 0).all()


def test_in_place_sum_other_stream_and_graph():
    from chunkwise_delta_rule_chunk_amd import binding as B
    from chunkwise_delta_rule_chunk_amd import ops
    x, r, w = _inputs(130, 2000, "bf16", "bf16", 4)
    want = ops.rms_norm(x, w, r)
    # the residual stream updated in place
    rr, y = r.clone(), torch.empty_like(x)
    d = B.RewyNormDesc(130, 2000, B.REWY_BF16, B.REWY_BF16, 0, 0, 1e-6, 0, 0, 0, 0)
    st = torch.cuda.current_stream().cuda_stream
    assert B.rewy_norm_fwd(d, x.data_ptr(), rr.data_ptr(), w.data_ptr(), rr.data_ptr(), y.data_ptr(), None, None,
                           None, st) == 0
    torch.cuda.synchronize()
    assert torch.equal(rr, want[1]) and torch.equal(y, want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.rms_norm(x, w, r, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    dy = torch.randn_like(x)
    ref = ops.rms_norm_backward(want[4], dy, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.rms_norm(x, w, r)
        gr = ops.rms_norm_backward(out[4], dy, x)
    for _ in range(3):
        out[0].zero_()
        gr["dx"].zero_()
        gr["dweight"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(gr["dx"], ref["dx"])
        assert torch.equal(gr["dweight"], ref["dweight"])


def test_autograd():
    from chunkwise_delta_rule_chunk_amd import ops
    x, r, w = (t.requires_grad_(True) for t in _inputs(17, 96, "fp32", "fp32", 2))
    y, s = ops.rms_norm_autograd(x, w, r, eps=EPS)
    (y.square().sum() + s.sum()).backward()
    xd, rd, wd = (t.detach().double().requires_grad_(True) for t in (x, r, w))
    sd, _, yd = _formula(xd, rd, wd)
    (yd.square().sum() + sd.sum()).backward()
    for a, b in ((x, xd), (r, rd), (w, wd)):
        assert (a.grad.double() - b.grad).norm() <= 1e-5 * b.grad.norm()


def test_more_rows_than_a_launch_has_threads():
    """2^28 + 5 short rows (over 2^32 threads): the first and the last rows are what they are alone."""
    from chunkwise_delta_rule_chunk_amd import ops
    M = (1 << 28) + 5
    x = torch.empty(M, 2, dtype=torch.bfloat16, device="cuda")
    x[:1000], x[-1000:] = 1.0, 3.0
    x[-1, 1] = -2.0
    y, _, _, _, ctx = ops.rms_norm(x)
    for cut in (slice(0, 1000), slice(M - 1000, M)):
        part = x[cut].contiguous()
        yp, _, _, _, cp = ops.rms_norm(part)
        assert torch.equal(y[cut], yp) and torch.equal(ctx["rstd"][cut], cp["rstd"])
