"""Group norm over a token's channels with a gate or an activation and the 8-bit
outputs, against the formula in 64 bits.

Bounds, U = 2^-24.  A group's sum takes at most L / 64 + 16 terms in a lane and 8
joining steps: k = L / 64 + 24.  The mean is within k U avg|x|, so x - mean within
e = U |x - mean| + k U avg|x|; the variance within k U of itself and what e brings to it
(at most 2 e rstd relative), rstd within half of that and 3 U, and xh = (x - mean) rstd
within rstd e + |xh| (k U + rstd max e + 4 U).  A sigmoid is within (2 |t| + 8) U of
itself for an argument t (the product with log2 e, the exponential, one sum, the
reciprocal); no activation is steeper than 1.1.  The backward is held to its own inputs,
mean and rstd as they were stored.  Outputs add half a step of their type."""
import pytest
import torch

from layer_util import DT, U32, close
from parity_util import gpu_available, say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

EPS = 1e-5


def act64(name, t):
    """value, derivative, bound of the derivative's derivative"""
    if name is None:
        return t, torch.ones_like(t)
    s = torch.sigmoid(t)
    return (s, s * (1 - s)) if name == "sigmoid" else (t * s, s * (1 + t * (1 - s)))


def inputs(M, G, L, dtype, wdt, seed, weight=True, bias=True, gate=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    D = G * L
    c = lambda t, d: t.to(d).cuda()  # noqa: E731
    x = rn(M, D) + 0.5
    x[:, seed % D] *= 10
    return (c(x, DT[dtype]), c(1 + 0.2 * rn(D), DT[wdt]) if weight else None, c(0.3 * rn(D), DT[wdt]) if bias else None,
            c(2 * rn(M, D), DT[dtype]) if gate else None, c(rn(M, D), DT[dtype]))


def forward64(x, w, b, z, G, center, act):
    """y and a bound of the fp32 arithmetic's error."""
    M, D = x.shape
    L = D // G
    k = L / 64 + 24
    x = x.double().view(M, G, L)
    mean = x.mean(-1, keepdim=True) if center else torch.zeros(M, G, 1, dtype=torch.float64, device=x.device)
    e = U32 * (x - mean).abs() + (k * U32 * x.abs().mean(-1, keepdim=True) if center else 0)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = (x - mean) * rstd
    err = rstd * e + xh.abs() * (k * U32 + rstd * e.amax(-1, keepdim=True) + 4 * U32)
    xh, err = xh.view(M, D), err.view(M, D)
    w = torch.ones((), dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros((), dtype=torch.float64, device=x.device) if b is None else b.double()
    n = xh * w + b
    err = err * w.abs() + 2 * U32 * ((xh * w).abs() + n.abs())
    t = n if z is None else z.double()
    a, _ = act64(act, t)
    rel = (2 * t.abs() + 10) * U32
    if z is None:
        return a, a.abs() * rel + 1.1 * err, mean, rstd
    return n * a, (n * a).abs() * (rel + U32) + a.abs() * err, mean, rstd


def backward64(x, w, b, z, mean, rstd, dy, G, center, act):
    """Gradients and bounds, from mean and rstd as stored."""
    M, D = x.shape
    L = D // G
    k = L / 64 + 24
    x, dy = x.double(), dy.double()
    rs = rstd.double().repeat_interleave(L, 1)
    mu = mean.double().repeat_interleave(L, 1) if center else 0.0
    xh = (x - mu) * rs
    wv = torch.ones((), dtype=torch.float64, device=x.device) if w is None else w.double()
    bv = torch.zeros((), dtype=torch.float64, device=x.device) if b is None else b.double()
    n = xh * wv + bv
    en = 4 * U32 * ((xh * wv).abs() + n.abs())
    t = n if z is None else z.double()
    a, da = act64(act, t)
    rel = (2 * t.abs() + 12) * U32
    s = torch.sigmoid(t) if act else torch.ones_like(t)
    # the derivative sums terms of both signs: s and s t (1 - s)
    da_mag = s * (1 + t.abs() * (1 - s)) if act else s
    if z is None:
        dn, edn = dy * da, dy.abs() * (da_mag * rel + 0.6 * en)
        dz = edz = None
    else:
        dn, edn = dy * a, (dy * a).abs() * rel
        dz, edz = dy * n * da, dy.abs() * (n.abs() * da_mag * rel + da.abs() * en)
    u, eu = dn * wv, edn * wv.abs() + U32 * (dn * wv).abs()
    grp = lambda v: v.view(M, G, L).mean(-1, keepdim=True).expand(M, G, L).reshape(M, D)  # noqa: E731
    c1 = grp(u) if center else torch.zeros_like(u)
    ec1 = grp(eu + k * U32 * u.abs()) if center else 0.0
    c2, ec2 = grp(u * xh), grp((eu + (k + 3) * U32 * u.abs()) * xh.abs())
    dx = rs * (u - c1 - xh * c2)
    edx = rs * (eu + ec1 + xh.abs() * ec2 + 6 * U32 * (u.abs() + c1.abs() + (xh * c2).abs()))
    terms, eterms = dn * xh, edn * xh.abs() + 4 * U32 * (dn * xh).abs()
    # at most M / 1024 + 1 rows in a register, then 16 + 64 joining steps
    rows = (M / 1024 + 100) * U32
    return (dict(dx=dx, dgate=dz, dweight=terms.sum(0) if w is not None else None,
                 dbias=dn.sum(0) if b is not None else None),
            dict(dx=edx, dgate=edz, dweight=eterms.sum(0) + rows * terms.abs().sum(0),
                 dbias=edn.sum(0) + rows * dn.abs().sum(0)))


SHAPES = [
    # M, G, L: groups in lanes of every width, whole rows, odd lengths, one channel, one group
    (1, 1, 1), (3, 2, 8), (5, 32, 4), (7, 3, 16), (33, 4, 32), (9, 5, 64), (257, 2, 128), (6, 32, 128), (4, 16, 256),
    (3, 7, 512), (5, 29, 53), (2, 1, 1537), (3, 1, 16384), (2, 16384, 1), (4, 3, 600), (70000, 1, 8), (2, 5, 1000),
    (1500, 3, 24), (3, 2, 1030), (2, 3, 5000), (4, 2, 4096), (5, 1, 5),
    # several waves a row and several rows a block, one group
    (7, 1, 1000), (6, 1, 500), (9, 1, 260), (5, 3, 300), (130, 1, 200), (3, 5, 40),
]


@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("M,G,L", SHAPES)
def test_forward_and_backward(M, G, L, dtype, wdt):
    from chunkwise_delta_rule_chunk_amd import ops
    v = M + 2 * G + 3 * L + (dtype == "bf16")
    center, gate, act = v % 2 == 0, v % 3 != 0, ("silu", "sigmoid", None)[v % 5 % 3]
    x, w, b, z, dy = inputs(M, G, L, dtype, wdt, v, v % 7 != 0, v % 4 != 0, gate)
    y, q, scale, ctx = ops.group_norm(x, w, b, z, groups=G, center=center, eps=EPS, activation=act)
    assert q is None and scale is None and (ctx["mean"] is not None) == center
    ref, err, mean, rstd = forward64(x, w, b, z, G, center, act)
    close(y, ref, err, "y")
    gr = ops.group_norm_backward(ctx, dy)
    ref, err = backward64(x, w, b, z, ctx["mean"], ctx["rstd"], dy, G, center, act)
    for k in ref:
        assert (gr[k] is None) == (ref[k] is None), k
        if gr[k] is not None:
            close(gr[k], ref[k], err[k], k)


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("act", ["silu", "sigmoid", None])
@pytest.mark.parametrize("L", [16, 11])
def test_backward_is_the_forwards_derivative(L, act, gate):
    """Gradients against central differences of the formula in 64 bits."""
    from chunkwise_delta_rule_chunk_amd import ops
    G = 3
    x, w, b, z, dy = inputs(3, G, L, "fp32", "fp32", 5, gate=gate)
    _, _, _, ctx = ops.group_norm(x, w, b, z, groups=G, eps=EPS, activation=act)
    gr = ops.group_norm_backward(ctx, dy)
    loss = lambda *t: (forward64(*t, G, True, act)[0] * dy.double()).sum().item()  # noqa: E731
    args = [None if t is None else t.double() for t in (x, w, b, z)]
    r = torch.Generator().manual_seed(2)
    for i, name in enumerate(("dx", "dweight", "dbias", "dgate")):
        if args[i] is None:
            continue
        d = torch.randn(args[i].shape, generator=r).double().cuda()
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        num = (loss(*up) - loss(*down)) / (2 * h)
        got = (gr[name].double() * d).sum().item()
        mag = (gr[name].double() * d).abs().sum().item()
        say(f"[layer] {name}: {got} against {num}")
        # differences: h^2 times a third derivative (below 1e3 of the magnitudes) and 2^-53 / h; fp32: 200 U
        assert abs(got - num) <= (1e-7 + 200 * U32) * mag + 1e-9


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("M,G,L,dtype", [(5, 4, 128, "bf16"), (3, 7, 11, "fp32"), (2, 3, 500, "bf16"), (4, 64, 4, "fp32"),
                                         (7, 8, 128, "bf16"), (5, 4, 200, "bf16"), (6, 3, 150, "fp32"), (67, 1, 32, "bf16"),
                                         (9, 1, 60, "bf16"), (11, 2, 100, "bf16"), (3, 1, 5000, "fp32")])
def test_codes(M, G, L, dtype, group, quant):
    """Scales from the unrounded y; codes are y over the stored scale, rounded once."""
    from chunkwise_delta_rule_chunk_amd import ops
    x, w, b, z, _ = inputs(M, G, L, dtype, dtype, group + L)
    D = G * L
    x[0] = 0  # a row of zeros: scale 1 where nothing else is added
    args = (x, w, None, z)
    y, q, scale, _ = ops.group_norm(*args, groups=G, eps=EPS, quant=quant, group=group)
    none, q2, scale2, _ = ops.group_norm(*args, groups=G, eps=EPS, quant=quant, group=group, output=False)
    assert none is None and torch.equal(scale, scale2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    y2, _, _, _ = ops.group_norm(*args, groups=G, eps=EPS)
    assert torch.equal(y, y2)
    ref, err, _, _ = forward64(*args, G, True, "silu")
    g = group or D
    ng = -(-D // g)
    pad = lambda t: torch.nn.functional.pad(t, (0, ng * g - D)).view(M, ng, g)  # noqa: E731
    top = 448.0 if quant == "e4m3" else 127.0
    amax, eamax = pad(ref).abs().amax(-1), pad(err).amax(-1)
    assert scale.shape == (M, ng)
    want = torch.where(amax < 2.0 ** -100, torch.ones_like(amax), amax / top)
    assert ((scale.double() - want).abs() <= eamax / top + 2 * U32 * want).all()
    full = scale.double().repeat_interleave(g, 1)[:, :D]
    val = q.double() * full
    # half a code's step, and the value's own error
    if quant == "int8":
        half = 0.5 * full
    else:
        half = torch.maximum((ref.abs() + err) * 2.0 ** -4, full * 2.0 ** -10)
    assert ((val - ref).abs() <= half + err + 2 * U32 * ref.abs()).all()
    assert (q[0].float() == 0).all()


def test_infinities_and_nans_stay_in_their_group():
    from chunkwise_delta_rule_chunk_amd import ops
    for L in (32, 11):
        x, w, b, z, _ = inputs(4, 6, L, "bf16", "bf16", 3)
        y0, _, s0, _ = ops.group_norm(x, w, b, z, groups=6, quant="e4m3", group=32)
        x[1, 2 * L + 3] = float("inf")
        x[2, 4 * L] = float("nan")
        y, _, s, _ = ops.group_norm(x, w, b, z, groups=6, quant="e4m3", group=32)
        hit = torch.zeros(4, 6 * L, dtype=torch.bool, device="cuda")
        hit[1, 2 * L:3 * L] = hit[2, 4 * L:5 * L] = True
        assert torch.equal(y[~hit], y0[~hit]) and not torch.isfinite(y[2, 4 * L:5 * L]).any()
        # a scale that covers a NaN is no finite number, the others stay
        ng = s.shape[1]
        cover = torch.nn.functional.pad(hit, (0, ng * 32 - 6 * L)).view(4, ng, 32).any(-1)
        assert torch.equal(s[~cover], s0[~cover]) and not torch.isfinite(s[2][cover[2]]).any()


def test_strided_rows_and_autograd():
    from chunkwise_delta_rule_chunk_amd import ops
    G, L = 4, 48
    row = torch.randn(2, 5, 3 * G * L, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    w, b = (torch.randn(G * L, generator=torch.Generator().manual_seed(i)).cuda().requires_grad_() for i in (1, 2))
    base = row.clone().requires_grad_()
    x, _, z = base.split(G * L, dim=-1)
    y = ops.group_norm_autograd(x, w, b, z, groups=G, eps=EPS)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    y.backward(dy)
    xs, zs = (t.detach().contiguous().flatten(0, 1) for t in (x, z))
    y2, _, _, ctx = ops.group_norm(xs, w.detach(), b.detach(), zs, groups=G, eps=EPS)
    g2 = ops.group_norm_backward(ctx, dy.flatten(0, 1))
    assert torch.equal(y.detach().flatten(0, 1), y2)
    gx, g0, gz = base.grad.flatten(0, 1).split(G * L, dim=-1)
    assert torch.equal(gx, g2["dx"]) and torch.equal(gz, g2["dgate"]) and (g0 == 0).all()
    assert torch.equal(w.grad, g2["dweight"]) and torch.equal(b.grad, g2["dbias"])
