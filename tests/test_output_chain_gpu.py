"""The attention with a constant decay, the group norm and the e4m3 product as a layer runs
them: norm to codes, product into one row of queries, keys, values and gate, attention on
slices of it, gated norm by head to codes, product; a prompt against the same tokens one by
one, a captured step, and the layer's gradients.

Bounds.  Gradients, 32 bits throughout: each operator is within 1e-5 of its 64-bit value in
norm (their own tests, where the attention's is the widest; measured below 1e-6), and a
gradient passes the attention twice (its inputs and its adjoint) and each norm and product
twice: 1e-5 for each of the four.  Serving in 16 bits: the row is off by at most
2^-8 + 1e-4 in norm on either side, the attention is linear in three of its parts and adds
2^-8: 2 (3 (2^-8 + 1e-4) + 2^-8) between the two sides for o, and the state without the
query and without the rounding of o: 4 (2^-8 + 1e-4).  A code stands for its value within 2^-4 on
either side, and the gate is a fourth part of the row: the sum of 2 (5 x 2^-8 + 4e-4), 2 x 2^-4 and
two roundings of the result."""
import pytest
import torch

from parity_util import gpu_available, say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

D, H, G, K, V = 256, 4, 2, 64, 64
CUTS = [H * K, G * K, G * V, H * V]
LOG_DECAY = [-0.7, -0.1, -0.02, -0.004]


def _codes(w):
    """w [N, K] as codes with a scale for each block of 128 x 128."""
    N, K = w.shape
    b = w.view(N // 128, 128, K // 128, 128)
    s = b.abs().amax((1, 3)) / 448
    return (b / s[:, None, :, None]).view(N, K).to(torch.float8_e4m3fn).cuda(), s.cuda()


def _weights():
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(n1=(1 + 0.1 * rn(D)).cuda(), n2=(1 + 0.1 * rn(H * V)).cuda(), wp=rn(sum(CUTS), D) * D ** -0.5,
                wo=rn(D, H * V) * (H * V) ** -0.5, g=torch.tensor(LOG_DECAY).cuda())


def _heads(row):
    q, k, v, z = row.split(CUTS, -1)
    return q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V)), z


def _serve(x, w, wp, wo, state, prompt, cu=None, inplace=False):
    from chunkwise_delta_rule_chunk_amd import ops
    _, _, c, s, _ = ops.rms_norm(x, w["n1"].bfloat16(), quant="e4m3", group=128, output=False)
    q, k, v, z = _heads(ops.e4m3_linear(c, s, *wp))
    if prompt:
        o, st, _ = ops.decay_attention(q, k, v, w["g"], h0=state, cu_seqlens=cu)
    else:
        o, st = ops.decay_attention_recurrent(q, k, v, w["g"], h0=state, ht=state if inplace else None)
    _, c, s, _ = ops.group_norm(o.flatten(2), w["n2"].bfloat16(), None, z, groups=H, center=False, quant="e4m3", group=128,
                                output=False)
    return ops.e4m3_linear(c, s, *wo), st, o


def _near(a, b, bound, what):
    rel = ((a.double() - b.double()).norm() / b.double().norm()).item()
    say(f"[layer] {what}: {rel:.2e} in norm, bound {bound:.2e}")
    assert rel <= bound, (what, rel)


@pytest.mark.parametrize("T", [1, 130, 300])
def test_a_prompt_and_its_tokens(T):
    w = _weights()
    wp, wo = _codes(w["wp"]), _codes(w["wo"])
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(2, T + 3, D, generator=g, device="cuda").bfloat16()
    state = torch.randn(2, H, K, V, generator=g, device="cuda")
    y, st, o = _serve(x, w, wp, wo, state, True)
    ys, os, s = [], [], state
    for t in range(T + 3):
        yt, s, ot = _serve(x[:, t:t + 1], w, wp, wo, s, False)
        ys.append(yt)
        os.append(ot)
    _near(torch.cat(os, 1), o, 2 * (4 * 2.0 ** -8 + 3e-4), "o")
    _near(s, st, 4 * (2.0 ** -8 + 1e-4), "state")
    last = 2 * (5 * 2.0 ** -8 + 4e-4) + 2 * 2.0 ** -4 + 2 * 2.0 ** -8
    _near(torch.cat(ys, 1), y, last, "output")
    # a prompt, its state, then tokens: and two prompts packed into one call
    _, mid, _ = _serve(x[:, :T].contiguous(), w, wp, wo, state, True)
    for t in range(T, T + 3):
        yt, mid, _ = _serve(x[:, t:t + 1], w, wp, wo, mid, False)
        _near(yt, y[:, t:t + 1], last, f"output of token {t}")
    cu = torch.tensor([0, T + 3, 2 * T + 6], dtype=torch.int32, device="cuda")
    yp, sp, _ = _serve(x.flatten(0, 1)[None], w, wp, wo, state, True, cu)
    _near(yp.view_as(y), y, last, "packed output")
    _near(sp, st, 4 * (2.0 ** -8 + 1e-4), "packed state")


def test_a_captured_step():
    """The step as a graph, its state updated in place: bit by bit the steps of the program."""
    w = _weights()
    wp, wo = _codes(w["wp"]), _codes(w["wo"])
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(6, 3, 1, D, generator=g, device="cuda").bfloat16()
    state = torch.randn(3, H, K, V, generator=g, device="cuda")
    want, s = [], state.clone()
    for t in range(6):
        y, _, _ = _serve(x[t], w, wp, wo, s, False, inplace=True)
        want.append(y)
    one, st = x[0].clone(), state.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, _ = _serve(one, w, wp, wo, st, False, inplace=True)
    for t in range(6):
        one.copy_(x[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[t]), t
    assert torch.equal(st, s)


def _layer64(x, w, h0, lens):
    n = lambda s, w, per: (s.unflatten(-1, (-1, per)) * (s.unflatten(-1, (-1, per)).square().mean(-1, keepdim=True)  # noqa: E731
                                                        + 1e-6).rsqrt()).flatten(-2) * w
    row = n(x, w["n1"], D) @ w["wp"].t()
    q, k, v, z = (t[0] for t in _heads(row))
    k, v = k.repeat_interleave(H // G, 1), v.repeat_interleave(H // G, 1)
    lam, os, sts, t0 = torch.exp(w["g"].double())[:, None, None], [], [], 0
    for i, ln in enumerate(lens):
        S = h0[i]
        for t in range(t0, t0 + ln):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            os.append((S * q[t][:, :, None]).sum(1) * K ** -0.5)
        sts.append(S)
        t0 += ln
    y = n(torch.stack(os)[None].flatten(2), w["n2"], V) * torch.nn.functional.silu(z)
    return y @ w["wo"].t(), torch.stack(sts)


@pytest.mark.parametrize("lens", [[150], [1, 70, 0, 79]])
def test_training(lens):
    from chunkwise_delta_rule_chunk_amd import ops
    T = sum(lens)
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, h0, dy, dst = rn(1, T, D), rn(len(lens), H, K, V), rn(1, T, D), rn(len(lens), H, K, V)
    w = {k: v.cuda() for k, v in _weights().items()}
    cu = None if len(lens) == 1 else torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda()
    names = ("n1", "n2", "wp", "wo")

    def leaves(dtype):
        f = lambda t: t.detach().to(dtype).requires_grad_(True)  # noqa: E731
        return f(x), f(h0), dict({k: f(w[k]) for k in names}, g=w["g"])
    x1, s1, w1 = leaves(torch.float32)
    y, _ = ops.rms_norm_autograd(x1, w1["n1"])
    q, k, v, z = _heads(y @ w1["wp"].t())
    o, st = ops.decay_attention_autograd(q, k, v, w1["g"], h0=s1, cu_seqlens=cu)
    n = ops.group_norm_autograd(o.flatten(2), w1["n2"], None, z, groups=H, center=False, eps=1e-6)
    out = n @ w1["wo"].t()
    x2, s2, w2 = leaves(torch.float64)
    ref, rst = _layer64(x2, w2, s2, lens)
    _near(out, ref, 4e-5, "output")
    _near(st, rst, 4e-5, "state")
    got = torch.autograd.grad((out * dy).sum() + (st * dst).sum(), [x1, s1, *(w1[k] for k in names)])
    want = torch.autograd.grad((ref * dy.double()).sum() + (rst * dst.double()).sum(), [x2, s2, *(w2[k] for k in names)])
    for a, b, k in zip(got, want, ("x", "h0", *names)):
        _near(a, b, 4e-5, "d" + k)
