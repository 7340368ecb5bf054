"""Shared helpers of the tests of the operators around the token mixer: plain
64-bit evaluations and element-wise error bounds."""
import torch

from parity_util import say

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, ref, slack, label):
    """|got - ref| <= half a step of got's type at ref + slack (a bound of the
    fp32 arithmetic's error, element by element), in 64 bits."""
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    u = half_step(got.dtype)
    g, r = got.double().cpu(), ref.double().cpu()
    slack = slack.double().cpu() if torch.is_tensor(slack) else torch.tensor(float(slack), dtype=torch.float64)
    # the value that is rounded lies within slack of ref (and bf16 and fp32 share their smallest step)
    bound = u * (r.abs() + slack) + slack + 1e-45
    if got.numel():
        over = ((g - r).abs() / bound)
        assert torch.isfinite(g).all(), f"{label}: not finite"
        worst = over.max().item()
        say(f"[layer] {label}: worst error {worst:.3f} of the bound")
        assert worst <= 1.0, f"{label}: error {worst:.2f} times the bound"


def scan_formula(x, dt, a_log, b, c, d, dt_bias, h0, lens, dy=None, dht=None):
    """The scan's definition token by token in 64 bits, all outputs and (with dy)
    all gradients by autograd, as a dict."""
    dev = x.device
    H, V = x.shape[-2:]
    G, K = b.shape[-2:]
    leaf = lambda t: None if t is None else t.detach().double().requires_grad_(dy is not None)  # noqa: E731
    n = len(lens)
    x64, dt64, b64, c64 = (leaf(t.flatten(0, 1)) for t in (x, dt, b, c))
    al, d64, bias = leaf(a_log), leaf(d), leaf(dt_bias)
    h64 = leaf(h0 if h0 is not None else torch.zeros(n, H, K, V, device=dev))
    ys, hts, t0 = [], [], 0
    for k, ln in enumerate(lens):
        S = h64[k]
        for t in range(t0, t0 + ln):
            z = dt64[t] + (0 if bias is None else bias)
            step = torch.nn.functional.softplus(z, threshold=80)
            bt, ct = (u[t].repeat_interleave(H // G, 0) for u in (b64, c64))
            S = torch.exp(-al.exp() * step)[:, None, None] * S + (step[:, None] * bt)[:, :, None] * x64[t][:, None, :]
            y = (S * ct[:, :, None]).sum(1)
            ys.append(y if d64 is None else y + d64[:, None] * x64[t])
        hts.append(S)
        t0 += ln
    y = torch.stack(ys) if ys else x64.new_zeros(0, H, V)
    ht = torch.stack(hts)
    out = dict(y=y.detach().reshape(x.shape), ht=ht.detach())
    if dy is None:
        return out
    loss = (y * dy.flatten(0, 1).double()).sum()
    if dht is not None:
        loss = loss + (ht * dht.double()).sum()
    names = dict(dx=x64, ddt=dt64, da_log=al, db=b64, dc=c64, dd=d64, ddt_bias=bias, dh0=h64)
    use = {k: v for k, v in names.items() if v is not None}
    gr = torch.autograd.grad(loss, list(use.values()), allow_unused=True)
    for (k, v), g in zip(use.items(), gr):
        out[k] = torch.zeros_like(v) if g is None else g
    out["dx"] = out["dx"].reshape(x.shape)
    out["ddt"] = out["ddt"].reshape(dt.shape)
    out["db"], out["dc"] = out["db"].reshape(b.shape), out["dc"].reshape(c.shape)
    return out
