"""The operators around the token mixer as a layer runs them: norm with the
residual, projection, convolution over x, B and C side by side, scan on slices of
its output, norm; forward, backward and token by token; and the same front before
the chunkwise delta rule.

Bounds: fp32 throughout the training chain; each operator is within 1e-6 of its
64-bit value in norm (their own tests), the projections sum at most 96 products
(96 U = 6e-6 at worst, about 1e-6 in norm), and a gradient passes each operator
twice: 1e-5 in norm.  The gradients of A_log and dt_bias are sums over the tokens of
terms c_t of both signs, each of them within that bound, |error of c_t| <= 1e-5 |c_t|, so
the sum is within 1e-5 sum |c_t| and not within 1e-5 of what the terms leave.  In bf16 each of the four stored stages rounds by at most 2^-8
relative to its values, and the recurrence and the norms do not amplify a uniformly
distributed error in norm: 4 x 2^-8."""
import pytest
import torch

import oracle
from parity_util import TOL, compare, gpu_available, say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

D, H, V, G, K, W = 96, 4, 32, 2, 32, 4
ROW = H * V + 2 * G * K


def _weights(dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = dict(n1=1 + 0.1 * rn(D), n2=1 + 0.1 * rn(H * V), wp=rn(D, ROW) * D ** -0.5, wd=rn(D, H) * D ** -0.5,
             cw=(torch.rand(ROW, W, generator=g) - 0.5), cb=0.1 * rn(ROW))
    w = {k: v.to(dtype) for k, v in w.items()}
    w.update(al=torch.log(1 + 7 * torch.rand(H, generator=g)), d=1 + 0.1 * rn(H), bias=rn(H) - 2)
    return {k: v.cuda() for k, v in w.items()}


def _slices(u):
    x, b, c = u.split([H * V, G * K, G * K], -1)
    return x.unflatten(-1, (H, V)), b.unflatten(-1, (G, K)), c.unflatten(-1, (G, K))


def _chain(x, r, w, cu):
    from chunkwise_delta_rule_chunk_amd import ops
    y, s = ops.rms_norm_autograd(x, w["n1"], r)
    u, _ = ops.short_conv_autograd(y @ w["wp"], w["cw"], w["cb"], cu_seqlens=cu)
    xs, b, c = _slices(u)
    o, ht = ops.selective_scan_autograd(xs, y @ w["wd"], w["al"], b, c, d=w["d"], dt_bias=w["bias"], cu_seqlens=cu)
    z, _ = ops.rms_norm_autograd(o.flatten(2), w["n2"])
    return z, s, ht


def _norm64(s, w):
    return s * (s.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w


def _chain64(x, r, w, lens):
    """w["al"] and w["bias"]: [T, H], a copy for each token."""
    s = x + r
    y = _norm64(s, w["n1"])
    u, dt, t0, us = (y @ w["wp"])[0], y @ w["wd"], 0, []
    for n in lens:
        ext = torch.cat([u.new_zeros(W - 1, ROW), u[t0:t0 + n]])
        us.append(torch.nn.functional.silu(sum(ext[j:j + n] * w["cw"][:, j] for j in range(W)) + w["cb"]))
        t0 += n
    xs, b, c = _slices(torch.cat(us)[None])
    ys, hts, t0 = [], [], 0
    for n in lens:
        S = x.new_zeros(H, K, V)
        for t in range(t0, t0 + n):
            step = torch.nn.functional.softplus(dt[0, t] + w["bias"][t], threshold=80)
            bt, ct = (q[0, t].repeat_interleave(H // G, 0) for q in (b, c))
            S = torch.exp(-w["al"][t].exp() * step)[:, None, None] * S + (step[:, None] * bt)[:, :, None] * xs[0, t][:, None]
            ys.append((S * ct[:, :, None]).sum(1) + w["d"][:, None] * xs[0, t])
        hts.append(S)
        t0 += n
    z = _norm64(torch.stack(ys)[None].flatten(2), w["n2"])
    return z, s, torch.stack(hts)


@pytest.mark.parametrize("lens", [[150], [1, 70, 0, 79]])
def test_training_chain(lens):
    T = sum(lens)
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, r, dz, dsum, dht = rn(1, T, D), rn(1, T, D), rn(1, T, H * V), rn(1, T, D), rn(len(lens), H, K, V)
    w = {k: v.requires_grad_(True) for k, v in _weights(torch.float32).items()}
    cu = None
    if len(lens) > 1:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    xg, rg = x.clone().requires_grad_(True), r.clone().requires_grad_(True)
    z, s, ht = _chain(xg, rg, w, cu)
    ((z * dz).sum() + (s * dsum).sum() + (ht * dht).sum()).backward()
    w64 = {k: v.detach().double() for k, v in w.items()}
    w64.update({k: w64[k].expand(T, H).clone() for k in ("al", "bias")})
    for v in w64.values():
        v.requires_grad_(True)
    x64, r64 = x.double().requires_grad_(True), r.double().requires_grad_(True)
    z64, s64, ht64 = _chain64(x64, r64, w64, lens)
    ((z64 * dz.double()).sum() + (s64 * dsum.double()).sum() + (ht64 * dht.double()).sum()).backward()
    errs = {}
    for name, a, b in [("z", z, z64), ("s", s, s64), ("ht", ht, ht64), ("dx", xg.grad, x64.grad), ("dr", rg.grad, r64.grad)] + \
            [("d" + k, w[k].grad, w64[k].grad) for k in w if k not in ("al", "bias")]:
        errs[name] = ((a.detach().double() - b).norm() / b.norm()).item()
    for k in ("al", "bias"):
        c = w64[k].grad
        errs["d" + k] = ((w[k].grad.double() - c.sum(0)).abs() / c.abs().sum(0)).max().item()
    say("[chain] " + " ".join(f"{k} {v:.1e}" for k, v in errs.items()))
    assert max(errs.values()) <= 1e-5


def test_prompt_and_tokens():
    """A prompt and then single tokens, all states carried, against the whole sequence as one prompt and in 64 bits."""
    from chunkwise_delta_rule_chunk_amd import ops
    n, T, P = 3, 45, 40
    g = torch.Generator().manual_seed(5)
    x, r = (torch.randn(n, T, D, generator=g).bfloat16().cuda() for _ in range(2))
    w = _weights(torch.bfloat16)
    kw = dict(d=w["d"], dt_bias=w["bias"])

    def front(a, b):
        y, s, _, _, _ = ops.rms_norm(a, w["n1"], b)
        return y @ w["wp"], y @ w["wd"]

    def back(o):
        return ops.rms_norm(o.flatten(-2), w["n2"], quant="e4m3")

    def prompt(a, b):
        u, dt = front(a, b)
        u, hc, _ = ops.short_conv(u, w["cw"], w["cb"], output_final_state=True)
        xs, bm, cm = _slices(u)
        o, hs, _ = ops.selective_scan(xs, dt, w["al"], bm, cm, **kw)
        return back(o)[0], hc, hs

    whole, hc_all, hs_all = prompt(x, r)
    z, hc, hs = prompt(x[:, :P].contiguous(), r[:, :P].contiguous())
    outs = [z]
    for t in range(P, T):
        u, dt = front(x[:, t], r[:, t])
        u, hc = ops.short_conv_step(u, hc, w["cw"], w["cb"], ht=hc)
        xs, bm, cm = _slices(u[:, None])
        o, hs = ops.selective_scan_recurrent(xs, dt[:, None], w["al"], bm, cm, **kw, h0=hs, ht=hs)
        z, _, q, scale, _ = back(o)
        assert ((q.float() * scale.view(n, 1, 1) - z.float()).abs() <= 2.0 ** -4 * z.float().abs() + 2.0 ** -9 * scale.view(n, 1, 1) + 2.0 ** -8 * z.float().abs()).all()
        outs.append(z)
    got = torch.cat(outs, 1).double()
    w64 = {k: v.double() for k, v in w.items()}
    w64.update({k: w64[k].expand(T, H) for k in ("al", "bias")})
    ref = torch.cat([_chain64(x[i:i + 1].double(), r[i:i + 1].double(), w64, [T])[0] for i in range(n)])
    for name, a in (("steps", got), ("prompt", whole.double())):
        rel = ((a - ref).norm() / ref.norm()).item()
        say(f"[chain] {name} {rel:.2e}")
        assert rel <= 4 * 2.0 ** -8
    assert ((hs - hs_all).norm() / hs_all.norm()).item() <= 4 * 2.0 ** -8
    assert (hc.float() - hc_all.float()).norm() <= 2.0 ** -7 * hc_all.float().norm()


def test_front_of_the_delta_rule():
    """Norm and convolution before the chunkwise delta rule: q, k, v are slices of the convolution's output."""
    from chunkwise_delta_rule_chunk_amd import ops
    T, heads, d = 100, 2, 64
    g = torch.Generator().manual_seed(9)
    x, r = (torch.randn(1, T, 192, generator=g).bfloat16().cuda() for _ in range(2))
    wp = (torch.randn(192, 3 * heads * d, generator=g) * 192 ** -0.5).bfloat16().cuda()
    cw = (torch.rand(3 * heads * d, W, generator=g) - 0.5).bfloat16().cuda()
    beta = torch.sigmoid(torch.randn(1, T, heads, generator=g)).bfloat16().cuda()
    gate = -torch.nn.functional.softplus(torch.randn(1, T, heads, generator=g) - 2).cuda()
    y, _, _, _, _ = ops.rms_norm(x, None, r)
    u, _, _ = ops.short_conv(y @ wp, cw)
    q, k, v = (t.unflatten(-1, (heads, d)).contiguous() for t in u.split(heads * d, -1))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).bfloat16() for t in (q, k))
    o, ht, _ = ops.forward(q, k, v, gate, beta)
    torch.cuda.synchronize()
    c = lambda t: t.cpu()  # noqa: E731
    ro, rht = oracle.forward(c(q), c(k), c(v), c(gate), c(beta), scale=d ** -0.5)
    compare(dict(o=o.double().cpu().numpy(), ht=ht.double().cpu().numpy()), dict(o=ro, ht=rht), TOL[torch.bfloat16],
            names=("o", "ht"), label="norm-conv-delta")
