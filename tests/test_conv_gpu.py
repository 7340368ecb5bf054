"""Short causal convolution (prompts, packed sequences, single tokens, backward)
against the formula in 64 bits.

Bounds.  pre sums W + 1 terms: (W + 2) U of their magnitudes (U = 2^-24, half a
step of fp32); the hardware's 2^x and reciprocal are within 2 U each, and SiLU's
slope is at most 1.1, so 16 U (|pre terms| + |y|) covers y.  dpre multiplies dy by
act'(pre), within 20 U (1 + |pre terms|).  Sums over tokens add half a step per
addition at most."""
import pytest
import torch

from layer_util import DT, U32, close
from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def _inputs(B, T, D, W, dtype, wdt, seed, nseq, bias=True, state=True):
    g = torch.Generator().manual_seed(seed)
    c = lambda t, d: t.to(d).cuda()  # noqa: E731
    x = c(torch.randn(B, T, D, generator=g), DT[dtype])
    w = c((torch.rand(D, W, generator=g) - 0.5) * 2, DT[wdt])
    b = c(torch.randn(D, generator=g) * 0.3, DT[wdt]) if bias else None
    h0 = c(torch.randn(nseq, W - 1, D, generator=g), DT[dtype]) if state else None
    dy = c(torch.randn(B, T, D, generator=g), DT[dtype])
    dht = c(torch.randn(nseq, W - 1, D, generator=g), DT[dtype]) if state else None
    return x, w, b, h0, dy, dht


def _formula(x, w, b, h0, dy, dht, silu, lens):
    """y, ht and all gradients in 64 bits, with the magnitudes that bound the fp32 error."""
    D, W = w.shape
    n = len(lens)
    leaf = lambda t: t.double().detach().requires_grad_(True)  # noqa: E731
    xs = leaf(x.reshape(-1, D))
    wd = leaf(w)
    bd = leaf(b) if b is not None else None
    hd = leaf(h0) if h0 is not None else torch.zeros(n, W - 1, D, dtype=torch.float64, device=x.device)
    ys, hts, mags, taps, t0 = [], [], [], [], 0
    for k, ln in enumerate(lens):
        ext = torch.cat([hd[k], xs[t0:t0 + ln]])
        pre = sum(ext[j:j + ln] * wd[:, j] for j in range(W))
        mag = sum((ext[j:j + ln] * wd[:, j]).abs() for j in range(W))
        if bd is not None:
            pre, mag = pre + bd, mag + bd.abs()
        ys.append(torch.nn.functional.silu(pre) if silu else pre)
        hts.append(ext[ln:])
        mags.append(mag)
        taps.append(torch.stack([ext[j:j + ln] for j in range(W)]))
        t0 += ln
    y, ht, mag = torch.cat(ys), torch.stack(hts), torch.cat(mags).detach()
    loss = (y * dy.reshape(-1, D).double()).sum()
    if dht is not None:
        loss = loss + (ht * dht.double()).sum()
    leaves = [xs, wd] + ([bd] if bd is not None else []) + ([hd] if h0 is not None else [])
    gr = list(torch.autograd.grad(loss, leaves))
    out = dict(y=y.detach(), ht=ht.detach(), dx=gr.pop(0), dweight=gr.pop(0),
               dbias=gr.pop(0) if bd is not None else None, dh0=gr.pop(0) if h0 is not None else None)
    # |dpre|'s bound and magnitudes of the sums over tokens
    dmag = dy.reshape(-1, D).double().abs() * (1 + mag) * 1.1
    out.update(mag=mag, dmag=dmag, tap=torch.cat(taps, 1).detach().abs())
    return out


def _check(got, ht, gr, ref, lens, w, dht):
    D, W = w.shape
    close(got.reshape(-1, D), ref["y"], 16 * U32 * (ref["mag"] + ref["y"].abs()), "y")
    if ht is not None:
        close(ht, ref["ht"], 0.0, "ht")
    if gr is None:
        return
    total, aw = sum(lens), w.double().abs()
    # dx_t: W taps of dpre, each within 20 U of its magnitude
    reach = torch.zeros(total + W, D, dtype=torch.float64, device=w.device)
    hreach = torch.zeros(len(lens), W - 1, D, dtype=torch.float64, device=w.device)
    t0 = 0
    for k, ln in enumerate(lens):
        for o in range(W):
            part = ref["dmag"][t0:t0 + ln] * aw[:, W - 1 - o]
            keep = min(o, ln)
            reach[t0:t0 + ln - keep] += part[keep:]
            for i in range(keep):  # token i reaches row i - o < 0 of the state
                hreach[k, W - 1 + i - o] += part[i]
        t0 += ln
    dh = 0 if dht is None else dht.double().abs().max()
    close(gr["dx"].reshape(-1, D), ref["dx"], 30 * U32 * (reach[:total] + dh), "dx")
    if ref["dh0"] is not None:
        close(gr["dh0"], ref["dh0"], 30 * U32 * (hreach + dh), "dh0")
    # a run has at most 64 tokens; then 3 joins, total / 256 / 16 tiles and 16 joins
    steps = 64 + 3 + total / 4096 + 16 + 30
    close(gr["dweight"], ref["dweight"], steps * U32 * (ref["dmag"] * ref["tap"]).sum(1).t(), "dweight")
    if ref["dbias"] is not None:
        close(gr["dbias"], ref["dbias"], steps * U32 * ref["dmag"].sum(0), "dbias")


CASES = [
    # B, T, D, W, dtype, wdt, lens (packed) or None, bias, state, activation
    (1, 1, 8, 4, "bf16", "bf16", None, True, True, "silu"),
    (2, 2, 33, 4, "fp32", "fp32", None, True, True, "silu"),
    (1, 3, 1, 3, "bf16", "fp32", None, False, True, None),
    (3, 130, 70, 4, "bf16", "bf16", None, True, False, "silu"),
    (1, 1000, 520, 4, "bf16", "fp32", None, True, True, "silu"),
    (2, 513, 257, 2, "fp32", "bf16", None, True, True, None),
    (1, 300, 129, 4, "bf16", "bf16", [0, 1, 2, 0, 3, 4, 90, 0, 200, 0], True, True, "silu"),
    (1, 300, 129, 3, "fp32", "fp32", [299, 1], False, True, "silu"),
    (1, 64, 40, 4, "bf16", "fp32", [1] * 64, True, True, "silu"),
    (1, 20000, 64, 4, "bf16", "fp32", [9999, 1, 10000], True, False, "silu"),
    (70, 5, 24, 4, "bf16", "bf16", None, True, True, "silu"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"b{c[0]}t{c[1]}d{c[2]}w{c[3]}{c[4]}{'p' if c[6] else ''}" for c in CASES])
def test_forward_and_backward(case):
    from chunkwise_delta_rule_chunk_amd import ops
    B, T, D, W, dtype, wdt, lens, bias, state, act = case
    cu = None
    if lens:
        assert sum(lens) == T
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        if T % 2:
            cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ln = lens or [T] * B
    x, w, b, h0, dy, dht = _inputs(B, T, D, W, dtype, wdt, T + D, len(ln), bias, state)
    y, ht, ctx = ops.short_conv(x, w, b, activation=act, h0=h0, cu_seqlens=cu, output_final_state=True)
    gr = ops.short_conv_backward(ctx, dy, dht)
    ref = _formula(x, w, b, h0, dy, dht, act == "silu", ln)
    _check(y, ht, gr, ref, ln, w, dht)


@pytest.mark.parametrize("dtype,wdt,W,D", [("bf16", "bf16", 4, 4352), ("fp32", "bf16", 3, 130), ("bf16", "fp32", 2, 7)])
def test_steps_continue_a_prompt(dtype, wdt, W, D):
    """A prompt and then token by token, the state in place, equals the whole prompt bit by bit."""
    from chunkwise_delta_rule_chunk_amd import ops
    x, w, b, h0, dy, dht = _inputs(5, 13, D, W, dtype, wdt, 3, 5)
    whole, last, _ = ops.short_conv(x, w, b, h0=h0, output_final_state=True)
    head, st, _ = ops.short_conv(x[:, :6].contiguous(), w, b, h0=h0, output_final_state=True)
    outs = [head]
    for t in range(6, 13):
        y, new = ops.short_conv_step(x[:, t], st, w, b, ht=st if t % 2 else None)
        st = new
        outs.append(y[:, None])
    assert torch.equal(torch.cat(outs, 1), whole) and torch.equal(st, last)
    _check(whole, last, None, _formula(x, w, b, h0, dy, dht, True, [13] * 5), [13] * 5, w, dht)


def test_strides_and_rows_behind_the_last_sequence():
    from chunkwise_delta_rule_chunk_amd import ops, binding as B
    x, w, b, h0, dy, dht = _inputs(2, 50, 96, 4, "bf16", "bf16", 6, 2)
    big = torch.randn(2, 50, 300, device="cuda").bfloat16()
    big[..., 101:197] = x
    y0, ht0, c0 = ops.short_conv(x, w, b, h0=h0, output_final_state=True)
    y1, ht1, c1 = ops.short_conv(big[..., 101:197], w, b, h0=h0, output_final_state=True)
    assert torch.equal(y0, y1) and torch.equal(ht0, ht1)
    big2 = torch.zeros(2, 50, 300, device="cuda").bfloat16()
    big2[..., 3:99] = dy
    g0, g1 = ops.short_conv_backward(c0, dy, dht), ops.short_conv_backward(c1, big2[..., 3:99], dht)
    for k in g0:
        assert torch.equal(g0[k], g1[k]), k
    # offsets that end before T: the rows behind are neither read nor written
    cu = torch.tensor([0, 20, 37], dtype=torch.int32, device="cuda")
    xs = x.reshape(1, 100, 96).clone()
    xs[:, 37:] = float("nan")
    y = torch.full_like(xs, 7.0)
    d = B.RewyConvDesc(1, 100, 96, 4, 2, cu.data_ptr(), None, B.REWY_BF16, B.REWY_BF16, B.REWY_ACT_SILU, 0, 0, 0)
    st = torch.cuda.current_stream().cuda_stream
    assert B.rewy_conv_fwd(d, xs.data_ptr(), w.data_ptr(), b.data_ptr(), h0.data_ptr(), y.data_ptr(), None, st) == 0
    torch.cuda.synchronize()
    want = ops.short_conv(xs[:, :37].contiguous(), w, b, h0=h0, cu_seqlens=cu)[0]
    assert torch.equal(y[:, :37], want) and (y[:, 37:] == 7).all()
    dx = torch.full_like(xs, 7.0)
    dys = dy.reshape(1, 100, 96)
    dw, db, dh0 = torch.empty_like(w), torch.empty_like(b), torch.empty_like(h0)
    ws = torch.empty(B.rewy_conv_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    assert B.rewy_conv_bwd(d, xs.data_ptr(), w.data_ptr(), b.data_ptr(), h0.data_ptr(), dys.data_ptr(), None,
                           dx.data_ptr(), dw.data_ptr(), db.data_ptr(), dh0.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert (dx[:, 37:] == 7).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_other_stream_graph_and_autograd():
    from chunkwise_delta_rule_chunk_amd import ops
    x, w, b, h0, dy, dht = _inputs(1, 700, 200, 4, "bf16", "fp32", 6, 1)
    y, ht, ctx = ops.short_conv(x, w, b, h0=h0, output_final_state=True)
    ref = ops.short_conv_backward(ctx, dy, dht)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.short_conv(x, w, b, h0=h0, stream=side)
    side.synchronize()
    assert torch.equal(got[0], y)
    cu = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = ops.short_conv(x, w, b, h0=h0, cu_seqlens=cu, output_final_state=True)
        gr = ops.short_conv_backward(o[2], dy, dht)
    for _ in range(3):
        o[0].zero_()
        for t in gr.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0], y) and all(torch.equal(gr[k], ref[k]) for k in ref)
    xf, wf, bf, hf = (t.detach().float().requires_grad_(True) for t in (x[:, :9, :6].contiguous(), w[:6], b[:6], h0[:, :, :6].contiguous()))
    ya, hta = ops.short_conv_autograd(xf, wf, bf, h0=hf)
    (ya * dy[:, :9, :6]).sum().backward(retain_graph=True)
    # against central differences in 64 bits
    def loss(xd):
        ext = torch.cat([hf.detach()[0].double(), xd[0]])
        pre = sum(ext[j:j + 9] * wf.detach().double()[:, j] for j in range(4)) + bf.detach().double()
        return (torch.nn.functional.silu(pre) * dy[0, :9, :6].double()).sum()
    h = 1e-5
    for t, c in ((0, 0), (4, 3), (8, 5)):
        e = torch.zeros(1, 9, 6, dtype=torch.float64, device="cuda")
        e[0, t, c] = h
        num = (loss(xf.detach().double() + e) - loss(xf.detach().double() - e)) / (2 * h)
        assert abs(num.item() - xf.grad[0, t, c].item()) < 1e-5 * max(1, abs(num.item()))
