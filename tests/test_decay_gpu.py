"""Linear attention with one constant decay for each head (chunked forward and
backward, token-serial form) against its definition in 64 bits.

Bounds.  Every output is a sum of products whose magnitudes the same definition
gives for the absolute values of the inputs ("abs" below; the decays stay).  U =
2^-24 is half a step of fp32, 2^-8 of bf16.
- fp32 arithmetic: a term passes a sum of at most 64 tokens and 128 state rows in
  matrix products, 4 roundings per chunk it crosses, and a few factors (powers of the
  decay are within 2 U of themselves); (300 + 4 chunks) U abs covers them.
- bf16 operands: a coefficient inside a chunk and an entering state are rounded
  once each, and a term of o, dq, dk or dv meets one of the two: 2^-8 (1 + 2^-8) abs;
  the walk's states take a token's row in two bf16 pieces, 2^-16 abs.  The states that
  are handed out keep 24 bits: only the fp32 bound."""
import pytest
import torch

from layer_util import DT, U32, close
from parity_util import gpu_available, say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def formula(q, k, v, g, h0, scale, lens, do=None, dht=None):
    """All pairs of tokens at once, sequence by sequence, in 64 bits; gradients by autograd."""
    grad = do is not None
    leaf = lambda t: None if t is None else t.detach().double().cpu().requires_grad_(grad)  # noqa: E731
    H, K = q.shape[2:]
    G, V = v.shape[2:]
    q64, k64, v64 = leaf(q), leaf(k), leaf(v)
    h64 = leaf(h0 if h0 is not None else torch.zeros(len(lens), H, K, V))
    g64 = g.detach().double().cpu()
    power = lambda n: torch.where(n == 0, torch.ones((), dtype=torch.float64),  # noqa: E731
                                  torch.exp(g64.view(-1, *[1] * n.dim()) * n.clamp_min(1).double()))
    qf, kf, vf = (t.flatten(0, 1).transpose(0, 1) for t in (q64, k64, v64))  # [H, tokens, K]
    kf, vf = kf.repeat_interleave(H // G, 0), vf.repeat_interleave(H // G, 0)
    os, hts, t0 = [], [], 0
    for n, ln in enumerate(lens):
        a, b, c = (t[:, t0:t0 + ln] for t in (qf, kf, vf))
        i = torch.arange(ln)
        D = power(i[:, None] - i).tril()
        os.append(scale * ((a @ b.transpose(1, 2)) * D @ c + power(i + 1)[..., None] * (a @ h64[n])))
        hts.append(power(torch.tensor(ln))[:, None, None] * h64[n] + (b * power(ln - 1 - i)[..., None]).transpose(1, 2) @ c)
        t0 += ln
    o, ht = torch.cat(os, 1).transpose(0, 1), torch.stack(hts)
    out = dict(o=o.detach().reshape(*q.shape[:3], V), ht=ht.detach())
    if grad:
        loss = (o * do.double().cpu().flatten(0, 1)).sum()
        if dht is not None:
            loss = loss + (ht * dht.double().cpu()).sum()
        out.update(zip(("dq", "dk", "dv", "dh0"), torch.autograd.grad(loss, (q64, k64, v64, h64))))
    return out


def inputs(B, T, H, G, K, V, dtype, seed, nseq, state=True, decay="usual", joint=False):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    c = lambda t, d: t.to(d).cuda()  # noqa: E731
    dt = DT[dtype]
    if joint:  # slices of one row
        row = c(rn(B, T, H * K + G * K + G * V), dt)
        q, k, v = row.split([H * K, G * K, G * V], dim=-1)
        q, k, v = q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V))
    else:
        q, k, v = c(rn(B, T, H, K), dt), c(rn(B, T, G, K), dt), c(rn(B, T, G, V), dt)
    g = {"usual": torch.log1p(-2.0 ** -(1 + 9 * torch.rand(H, generator=gen))), "none": torch.zeros(H),
         "strong": -5.0 - 40 * torch.rand(H, generator=gen), "zero": torch.full((H,), -torch.inf)}[decay]
    h0 = c(0.5 * rn(nseq, H, K, V), torch.float32) if state else None
    do = c(rn(B, T, H, V), dt)
    dht = c(0.3 * rn(nseq, H, K, V), torch.float32) if state else None
    return (q, k, v, c(g, torch.float32)), h0, do, dht


def magnitudes(args, h0, scale, lens, do, dht):
    ab = lambda t: None if t is None else t.abs()  # noqa: E731
    q, k, v, g = args
    return formula(q.abs(), k.abs(), v.abs(), g, ab(h0), abs(scale), lens, ab(do), ab(dht))


def check(got, ref, mag, longest, dtype, names):
    fp = (300 + 4 * (longest / 64 + 1)) * U32
    op = 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -16 if dtype == "bf16" else 0.0
    for k in names:
        if got[k] is None:
            continue
        state = k in ("ht", "dh0")
        close(got[k], ref[k], (fp + (0 if state else op)) * mag[k], k)
        if got[k].numel() > 1000 and not state:
            rel = ((got[k].double().cpu() - ref[k]).norm() / ref[k].norm()).item()
            say(f"[layer] {k} norm error {rel:.2e}")
            # at most three independent roundings of relative size 2^-8 / sqrt(3) each
            assert rel <= (2.0 ** -8 if dtype == "bf16" else 1e-5)


CASES = [
    # B, T, H, G, K, V, dtype, lens, state, decay, joint row
    (1, 1, 1, 1, 32, 32, "bf16", None, True, "usual", False),
    (2, 63, 2, 1, 64, 32, "bf16", None, True, "usual", True),
    (1, 64, 3, 3, 32, 64, "fp32", None, False, "usual", False),
    (1, 65, 4, 2, 64, 64, "fp32", None, True, "usual", True),
    (1, 130, 6, 2, 128, 64, "bf16", None, True, "usual", True),
    (1, 200, 4, 4, 128, 128, "bf16", None, True, "usual", False),
    (2, 700, 2, 1, 64, 128, "bf16", None, True, "usual", True),
    (1, 600, 3, 1, 64, 32, "fp32", None, True, "usual", False),
    (1, 300, 2, 1, 128, 128, "fp32", None, True, "usual", True),
    (1, 300, 2, 2, 32, 128, "fp32", None, True, "none", False),
    (1, 300, 2, 2, 128, 32, "bf16", None, True, "strong", False),
    (1, 300, 2, 1, 128, 32, "fp32", None, True, "zero", False),
    (1, 300, 2, 1, 32, 128, "bf16", None, True, "none", True),
    (1, 600, 2, 2, 32, 32, "bf16", [0, 1, 64, 65, 0, 0, 300, 127, 43, 0], True, "usual", False),
    (1, 900, 3, 1, 64, 64, "fp32", [299, 1, 600], True, "usual", True),
    (1, 40, 4, 4, 128, 64, "bf16", [1] * 40, False, "usual", False),
    (1, 1100, 2, 1, 128, 128, "bf16", [700, 0, 400], True, "usual", True),
    (3, 0, 2, 1, 64, 64, "bf16", None, True, "usual", False),
]


@pytest.mark.parametrize("B,T,H,G,K,V,dtype,lens,state,decay,joint", CASES)
def test_forward_and_backward(B, T, H, G, K, V, dtype, lens, state, decay, joint):
    from chunkwise_delta_rule_chunk_amd import ops
    nseq = B if lens is None else len(lens)
    args, h0, do, dht = inputs(B, T, H, G, K, V, dtype, T + H + K + V, nseq, state, decay, joint)
    each = lens or [T] * B
    scale = K ** -0.5
    ref = formula(*args, h0, scale, each, do, dht)
    mag = magnitudes(args, h0, scale, each, do, dht)
    cu = None
    if lens:
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o, ht, ctx = ops.decay_attention(*args, h0=h0, cu_seqlens=cu)
    check(dict(o=o, ht=ht), ref, mag, max(each), dtype, ("o", "ht"))
    o2, none, _ = ops.decay_attention(*args, h0=h0, cu_seqlens=cu, output_final_state=False)
    assert none is None and torch.equal(o, o2)  # o does not depend on whether ht is given
    gr = ops.decay_attention_backward(ctx, do, dht, want_dh0=True)
    check(gr, ref, mag, max(each), dtype, ("dq", "dk", "dv", "dh0"))
    o3, ht3 = ops.decay_attention_recurrent(*args, h0=h0, cu_seqlens=cu)
    # a term's state takes three roundings a token
    fp = (300 + 4 * max(each)) * U32
    close(o3, ref["o"], fp * mag["o"], "o, token by token")
    close(ht3, ref["ht"], fp * mag["ht"], "ht, token by token")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_with_and_without_the_forwards_states(dtype):
    """A caller's own workspace is not kept: the states are formed again, bit by bit the same."""
    from chunkwise_delta_rule_chunk_amd import binding as B
    from chunkwise_delta_rule_chunk_amd import ops
    args, h0, do, dht = inputs(2, 700, 3, 1, 64, 64, dtype, 5, 2)
    o, ht, ctx = ops.decay_attention(*args, h0=h0)
    ws = torch.empty(B.rewy_decay_workspace_bytes(ctx["desc"], 0), dtype=torch.uint8, device="cuda")
    o2, ht2, ctx2 = ops.decay_attention(*args, h0=h0, ws=ws)
    assert ctx["states"] is not None and ctx2["states"] is None
    ws.fill_(255)
    assert torch.equal(o, o2) and torch.equal(ht, ht2)
    a, b = ops.decay_attention_backward(ctx, do, dht), ops.decay_attention_backward(ctx2, do, dht)
    assert all(torch.equal(a[k], b[k]) for k in a)
