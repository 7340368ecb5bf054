"""Selective state space scan (chunked forward and backward, token-serial form)
against its definition in 64 bits.

Bounds.  Every output is a sum of products whose magnitudes the same definition
gives for the absolute values of the inputs ("abs" below; the decays stay).  U =
2^-24 is half a step of fp32, 2^-8 of bf16.
- fp32 arithmetic: a term passes a sum of at most 64 tokens and 128 state rows in
  matrix products, up to 2 roundings per chunk it crosses and exponentials whose
  exponents are sums of 64 terms; (300 + 4 chunks) U abs covers them.
- bf16 operands: a coefficient inside a chunk and an entering state are rounded
  once each, and a term meets one of the two: 2^-8 (1 + 2^-8) abs, for y, dx, db,
  dc.  The states and everything that sums into ht, dh0, ddt and the parameters'
  gradients keep 24 bits: only the fp32 bound.
- ddt_t = (c_t + A dg_t) sigmoid: dg_t is a suffix sum whose terms' magnitudes are at
  most R_t = sum_{i >= t} (|r_i| + dt_i |c_i|) + <|S|, |dht|> (what the later tokens
  read of the state at t)."""
import pytest
import torch

from layer_util import DT, U32, close, scan_formula
from parity_util import gpu_available, say

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def _inputs(B, T, H, G, K, V, dtype, dtd, seed, nseq, state=True, decay="usual", skip=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = lambda t, d: t.to(d).cuda()  # noqa: E731
    step = {"usual": -3.0, "strong": 3.0, "none": -18.0}[decay]
    kw = dict(d=c(1 + 0.3 * rn(H), torch.float32) if skip else None, dt_bias=c(step + 0.5 * rn(H), torch.float32),
              h0=c(0.5 * rn(nseq, H, K, V), torch.float32) if state else None)
    args = (c(rn(B, T, H, V), DT[dtype]), c(rn(B, T, H), DT[dtd]),
            c(torch.log(1 + 15 * torch.rand(H, generator=g)), torch.float32), c(rn(B, T, G, K), DT[dtype]),
            c(rn(B, T, G, K), DT[dtype]))
    dy = c(rn(B, T, H, V), DT[dtype])
    dht = c(0.3 * rn(nseq, H, K, V), torch.float32) if state else None
    return args, kw, dy, dht


def _abs(t):
    return None if t is None else t.abs()


def _references(args, kw, lens, dy, dht):
    x, dt, al, b, c = args
    ref = scan_formula(x, dt, al, b, c, kw["d"], kw["dt_bias"], kw["h0"], lens, dy, dht)
    mag = scan_formula(x.abs(), dt, al, b.abs(), c.abs(), _abs(kw["d"]), kw["dt_bias"], _abs(kw["h0"]), lens,
                       _abs(dy), _abs(dht))
    return ref, mag


def _check_forward(y, ht, ref, mag, T, dtype):
    fp = (300 + 4 * (T / 64 + 1)) * U32
    op = 2.0 ** -8 * (1 + 2.0 ** -8) if dtype == "bf16" else 0.0
    close(y, ref["y"], (fp + op) * mag["y"], "y")
    if ht is not None:
        close(ht, ref["ht"], fp * mag["ht"], "ht")
    if y.numel() > 1000:
        rel = ((y.double() - ref["y"]).norm() / ref["y"].norm()).item()
        say(f"[layer] y norm error {rel:.2e}")
        # at most three independent roundings of relative size 2^-8 / sqrt(3) each
        assert rel <= (3 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 if dtype == "bf16" else 1e-5)


def _check_backward(gr, ref, mag, args, kw, lens, dy, dht, dtype):
    x, dt, al, b, c = args
    H = x.shape[2]
    fp = (300 + 4 * (max(lens) / 64 + 1)) * U32
    op = 2.0 ** -8 * (1 + 2.0 ** -8) if dtype == "bf16" else 0.0
    for k in ("dx", "db", "dc"):
        close(gr[k], ref[k], (fp + op) * mag[k], k)
        if gr[k].numel() > 1000:
            rel = ((gr[k].double() - ref[k]).norm() / ref[k].norm()).item()
            say(f"[layer] {k} norm error {rel:.2e}")
            assert rel <= (2.0 ** -8 if dtype == "bf16" else 1e-5)
    if gr["dh0"] is not None:
        close(gr["dh0"], ref["dh0"], fp * mag["dh0"], "dh0")
    # magnitudes of r and c, and R_t
    z = dt.double() + kw["dt_bias"].double()
    step = torch.nn.functional.softplus(z, threshold=80).flatten(0, 1)
    da = 0 if kw["d"] is None else kw["d"].double().abs()[:, None]
    ax, ady = x.double().abs().flatten(0, 1), dy.double().abs().flatten(0, 1)
    r = (ady * (mag["y"].flatten(0, 1) - da * ax)).sum(-1)
    stepc = (ax * (mag["dx"].flatten(0, 1) - da * ady)).sum(-1)  # dt c
    A = al.double().exp()
    R = torch.zeros_like(r)
    t0 = 0
    for k, ln in enumerate(lens):
        s = r[t0:t0 + ln] + stepc[t0:t0 + ln]
        tail = 0 if dht is None else (mag["ht"][k] * dht[k].double().abs()).sum((-1, -2))
        R[t0:t0 + ln] = s.flip(0).cumsum(0).flip(0) + tail
        t0 += ln
    slack = fp * (stepc / step + A * R)
    close(gr["ddt"].flatten(0, 1), ref["ddt"].flatten(0, 1), slack, "ddt")
    close(gr["ddt_bias"], ref["ddt_bias"], slack.sum(0), "ddt_bias")
    close(gr["da_log"], ref["da_log"], (fp * A * step * R).sum(0), "da_log")
    if kw["d"] is not None:
        close(gr["dd"], ref["dd"], fp * (ax * ady).sum((0, 2)), "dd")
    say(f"[layer] relative: " + " ".join(
        f"{k} {((gr[k].double() - ref[k]).norm() / ref[k].norm()).item():.1e}" for k in ("ddt", "ddt_bias", "da_log")))


CASES = [
    # B, T, H, G, K, V, dtype, dt dtype, lens, state, decay
    (1, 1, 1, 1, 32, 32, "bf16", "bf16", None, True, "usual"),
    (2, 63, 2, 1, 64, 32, "bf16", "fp32", None, True, "usual"),
    (1, 64, 3, 3, 32, 64, "fp32", "fp32", None, False, "usual"),
    (1, 65, 4, 2, 64, 64, "fp32", "bf16", None, True, "usual"),
    (1, 130, 5, 1, 128, 64, "bf16", "fp32", None, True, "usual"),
    (1, 200, 6, 2, 128, 128, "bf16", "bf16", None, True, "usual"),
    (2, 700, 2, 1, 64, 128, "bf16", "fp32", None, True, "usual"),
    (1, 600, 3, 1, 64, 32, "fp32", "fp32", None, True, "usual"),
    (1, 300, 2, 1, 32, 128, "bf16", "fp32", None, True, "strong"),
    (1, 300, 2, 1, 128, 32, "bf16", "fp32", None, True, "none"),
    (1, 600, 2, 2, 32, 32, "bf16", "fp32", [0, 1, 64, 65, 0, 0, 300, 127, 43, 0], True, "usual"),
    (1, 900, 3, 1, 64, 64, "fp32", "fp32", [299, 1, 600], True, "usual"),
    (1, 40, 4, 4, 128, 64, "bf16", "bf16", [1] * 40, False, "usual"),
    # one head a workgroup, and head blocks that a group does not fill, of every width
    (1, 100, 2, 2, 128, 32, "bf16", "fp32", None, True, "usual"),
    (1, 300, 5, 1, 32, 32, "bf16", "bf16", None, True, "usual"),
    (1, 300, 9, 3, 64, 64, "bf16", "fp32", None, True, "usual"),
    (2, 300, 3, 1, 32, 32, "fp32", "bf16", None, True, "usual"),
    (1, 520, 2, 2, 64, 32, "fp32", "fp32", [520], False, "none"),
    # several segments without a chunk that decays strongly, so that the decay gradient's
    # chains start at segment ends, from behind and from the front, with and without a state
    (1, 1100, 2, 1, 64, 64, "bf16", "fp32", None, False, "none"),
    (1, 1200, 2, 1, 32, 32, "bf16", "fp32", [700, 500], True, "none"),
]


def _cu(lens, T):
    if not lens:
        return None
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    assert cu[-1] == T
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("case", CASES, ids=["_".join(str(v) for v in c[:8]) + ("_packed" if c[8] else "") + "_" + c[10]
                                             for c in CASES])
def test_chunked_forward_and_backward(case):
    from chunkwise_delta_rule_chunk_amd import ops
    B, T, H, G, K, V, dtype, dtd, lens, state, decay = case
    say(f"[case] {case}")
    ln = lens or [T] * B
    args, kw, dy, dht = _inputs(B, T, H, G, K, V, dtype, dtd, T + K + V, len(ln), state, decay, skip=H != 3)
    y, ht, ctx = ops.selective_scan(*args, **kw, cu_seqlens=_cu(lens, T))
    torch.cuda.synchronize()
    ref, mag = _references(args, kw, ln, dy, dht)
    _check_forward(y, ht, ref, mag, max(ln), dtype)
    gr = ops.selective_scan_backward(ctx, dy, dht)
    torch.cuda.synchronize()
    _check_backward(gr, ref, mag, args, kw, ln, dy, dht, dtype)


@pytest.mark.parametrize("case", [
    (3, 1, 4, 2, 128, 64, "bf16", "bf16", None), (2, 5, 3, 3, 64, 128, "bf16", "fp32", None),
    (1, 9, 2, 1, 32, 32, "fp32", "fp32", [0, 4, 5, 0]), (1, 3, 2, 1, 128, 128, "bf16", "fp32", None),
    (2, 2, 2, 1, 64, 64, "fp32", "bf16", None), (1, 4, 2, 1, 32, 128, "bf16", "fp32", None)])
def test_token_serial_form(case):
    from chunkwise_delta_rule_chunk_amd import ops
    B, T, H, G, K, V, dtype, dtd, lens = case
    say(f"[case] {case}")
    ln = lens or [T] * B
    args, kw, dy, _ = _inputs(B, T, H, G, K, V, dtype, dtd, 5, len(ln))
    y, ht = ops.selective_scan_recurrent(*args, **kw, cu_seqlens=_cu(lens, T))
    ref, mag = _references(args, kw, ln, dy, None)
    fp = (300 + 4 * T) * U32
    close(y, ref["y"], fp * mag["y"], "y")
    close(ht, ref["ht"], fp * mag["ht"], "ht")
    # the state in place
    kw2 = dict(kw, h0=kw["h0"].clone())
    y2, ht2 = ops.selective_scan_recurrent(*args, **kw2, cu_seqlens=_cu(lens, T), ht=kw2["h0"])
    assert torch.equal(y, y2) and torch.equal(ht, ht2) and ht2 is kw2["h0"]


def test_prompt_then_single_tokens():
    """A chunked prompt, then single tokens from its state, against the whole definition."""
    from chunkwise_delta_rule_chunk_amd import ops
    args, kw, dy, _ = _inputs(2, 140, 4, 2, 64, 64, "bf16", "fp32", 9, 2)
    cut = lambda a, s: tuple(t[:, s].contiguous() if t.dim() > 1 else t for t in a)  # noqa: E731
    y, st, _ = ops.selective_scan(*cut(args, slice(0, 136)), **kw)
    outs = [y]
    for t in range(136, 140):
        y, st = ops.selective_scan_recurrent(*cut(args, slice(t, t + 1)), **dict(kw, h0=st))
        outs.append(y)
    ref, mag = _references(args, kw, [140, 140], dy, None)
    _check_forward(torch.cat(outs, 1), st, ref, mag, 140, "bf16")


def test_slices_of_one_row_and_rows_behind_the_last_sequence():
    """x, B, C as slices of the convolution's row and the gradients into slices of one row: bit by bit the
    contiguous results; offsets that end before T leave the rows behind alone."""
    from chunkwise_delta_rule_chunk_amd import ops
    B, T, H, G, K, V = 1, 333, 4, 2, 64, 32
    args, kw, dy, dht = _inputs(B, T, H, G, K, V, "bf16", "fp32", 2, 2)
    x, dt, al, b, c = args
    row = torch.cat([t.flatten(2) for t in (x, b, c)], -1)
    xs, bs, cs = (t.unflatten(-1, s) for t, s in zip(row.split([H * V, G * K, G * K], -1), ((H, V), (G, K), (G, K))))
    cu = torch.tensor([0, 100, 333], dtype=torch.int32, device="cuda")
    y0, ht0, c0 = ops.selective_scan(*args, **kw, cu_seqlens=cu)
    y1, ht1, c1 = ops.selective_scan(xs, dt, al, bs, cs, **kw, cu_seqlens=cu)
    assert torch.equal(y0, y1) and torch.equal(ht0, ht1)
    g0 = ops.selective_scan_backward(c0, dy, dht)
    drow = torch.full_like(row, 5.0)
    out = tuple(t.unflatten(-1, s) for t, s in zip(drow.split([H * V, G * K, G * K], -1), ((H, V), (G, K), (G, K))))
    g1 = ops.selective_scan_backward(c1, dy, dht, out=out)
    for k in g0:
        assert torch.equal(g0[k], g1[k]), k
    # the last 133 rows belong to no sequence
    cut = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    bad = row.clone()
    bad[:, 200:] = float("nan")
    xs, bs, cs = (t.unflatten(-1, s) for t, s in zip(bad.split([H * V, G * K, G * K], -1), ((H, V), (G, K), (G, K))))
    short = tuple(t[:, :200].contiguous() for t in (x, dt)) + (al,) + tuple(t[:, :200].contiguous() for t in (b, c))
    yw, htw, cw = ops.selective_scan(*short, **kw, cu_seqlens=cut)
    gw = ops.selective_scan_backward(cw, dy[:, :200].contiguous(), dht)
    y2, ht2, c2 = ops.selective_scan(xs, dt, al, bs, cs, **kw, cu_seqlens=cut)
    drow.fill_(5.0)
    g2 = ops.selective_scan_backward(c2, dy, dht, out=out)
    # (the cut into segments follows T, so sums over tokens may differ in their last bits)
    assert torch.isfinite(y2[:, :200]).all() and (y2[:, :200].float() - yw.float()).abs().max() <= 2.0 ** -6 * yw.float().abs().max()
    assert (ht2 - htw).abs().max() <= 1e-5 * htw.abs().max()
    assert (drow[:, 200:] == 5).all()
    for k in ("da_log", "dd", "ddt_bias", "dh0"):
        assert (g2[k] - gw[k]).norm() <= 1e-5 * gw[k].norm(), k


def test_same_result_every_time_other_stream_and_graph():
    from chunkwise_delta_rule_chunk_amd import ops
    args, kw, dy, dht = _inputs(1, 900, 4, 1, 128, 64, "bf16", "bf16", 4, 1)
    y, ht, ctx = ops.selective_scan(*args, **kw)
    gr = ops.selective_scan_backward(ctx, dy, dht)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, ht1, ctx1 = ops.selective_scan(*args, **kw, stream=side)
    g1 = ops.selective_scan_backward(ctx1, dy, dht, stream=side)
    side.synchronize()
    assert torch.equal(y, y1) and torch.equal(ht, ht1) and all(torch.equal(gr[k], g1[k]) for k in gr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, htg, cg = ops.selective_scan(*args, **kw)
        gg = ops.selective_scan_backward(cg, dy, dht)
        yr, htr = ops.selective_scan_recurrent(*args, **kw)
    rec = ops.selective_scan_recurrent(*args, **kw)
    for _ in range(3):
        for t in (yg, htg, yr, *gg.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and torch.equal(htg, ht) and all(torch.equal(gr[k], gg[k]) for k in gr)
        assert torch.equal(yr, rec[0]) and torch.equal(htr, rec[1])


def test_gradients_against_differences():
    from chunkwise_delta_rule_chunk_amd import ops
    args, kw, dy, dht = _inputs(1, 20, 2, 1, 32, 32, "fp32", "fp32", 8, 1)
    leaves = [t.requires_grad_(True) for t in (*args, kw["d"], kw["dt_bias"], kw["h0"])]
    y, ht = ops.selective_scan_autograd(*args, **kw)
    ((y * dy).sum() + (ht * dht).sum()).backward()

    def loss(vals):
        o = scan_formula(*vals[:5], vals[5], vals[6], vals[7], [20])
        return ((o["y"] * dy.double()).sum() + (o["ht"] * dht.double()).sum()).item()

    base = [t.detach().double() for t in leaves]
    h = 1e-5
    for i, t in enumerate(leaves):
        for pos in (0, t.numel() // 2, t.numel() - 1):
            up, dn = [v.clone() for v in base], [v.clone() for v in base]
            up[i].view(-1)[pos] += h
            dn[i].view(-1)[pos] -= h
            num = (loss(up) - loss(dn)) / (2 * h)
            got = t.grad.reshape(-1)[pos].item()
            assert abs(num - got) <= 2e-5 * max(1.0, abs(num), t.grad.abs().max().item()), (i, pos, num, got)


def test_no_tokens_and_one_long_sequence():
    from chunkwise_delta_rule_chunk_amd import ops
    args, kw, dy, dht = _inputs(2, 0, 2, 1, 32, 64, "bf16", "fp32", 8, 2)
    y, ht, ctx = ops.selective_scan(*args, **kw)
    assert y.shape[1] == 0 and torch.equal(ht, kw["h0"])
    gr = ops.selective_scan_backward(ctx, dy, dht)
    assert torch.equal(gr["dh0"], dht) and (gr["da_log"] == 0).all() and (gr["dd"] == 0).all()
    y, ht = ops.selective_scan_recurrent(*args, **kw)
    assert torch.equal(ht, kw["h0"])
    # a sequence alone and beside others: the same rows
    args, kw, dy, dht = _inputs(1, 3000, 2, 1, 64, 64, "bf16", "fp32", 3, 1)
    y, ht, ctx = ops.selective_scan(*args, **kw)
    yr, htr = ops.selective_scan_recurrent(*args, **kw)
    assert (ht - htr).norm() <= 1e-5 * htr.norm()
    assert (y.float() - yr.float()).norm() <= 2.0 ** -7 * yr.float().norm()


@pytest.mark.parametrize("K,V,H,dtype", [(128, 128, 2, "bf16"), (64, 64, 3, "bf16"), (32, 32, 5, "bf16"), (64, 32, 3, "fp32")])
def test_not_finite_values_reach_no_earlier_token(K, V, H, dtype):
    """A padded batch whose rows behind a row's tokens hold anything: y before them as without; y of the
    column from the first such x on is not finite."""
    from chunkwise_delta_rule_chunk_amd import ops
    B, T = 3, 150
    args, kw, _, _ = _inputs(B, T, H, 1, K, V, dtype, "fp32", 11, B)
    y0, _, _ = ops.selective_scan(*args, **kw)
    x, dt, al, b, c = (t.clone() for t in args)
    ends = [149, 65, 3]
    for n, (e, bad) in enumerate(zip(ends, (float("nan"), float("inf"), -float("inf")))):
        for t in (x, dt, b, c):
            t[n, e:] = bad
    y1, _, _ = ops.selective_scan(x, dt, al, b, c, **kw)
    for n, e in enumerate(ends):
        assert torch.equal(y0[n, :e], y1[n, :e])
    # one value of x only: its column from its token on, and nothing else
    x = args[0].clone()
    x[1, 70, 1, 5], x[1, 20, 1, 6] = float("inf"), float("nan")
    y2, h2, _ = ops.selective_scan(x, *args[1:], **kw)
    same = torch.ones_like(y0, dtype=torch.bool)
    same[1, 70:, 1, 5] = same[1, 20:, 1, 6] = False
    assert torch.equal(y2[same], y0[same]) and not torch.isfinite(y2[~same]).any()
    bad = torch.zeros_like(h2, dtype=torch.bool)
    bad[1, 1, :, 5:7] = True
    assert torch.equal(~torch.isfinite(h2), bad)


def test_autograd_clears_rows_behind_the_last_sequence():
    """Offsets that only the GPU holds may end before T: such rows have zero gradients, whatever the
    allocator's memory held."""
    from chunkwise_delta_rule_chunk_amd import ops
    args, kw, _, _ = _inputs(1, 90, 2, 1, 32, 32, "bf16", "fp32", 5, 1)
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    leaves = [t.requires_grad_(True) for t in (*args, kw["h0"])]
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
    del junk
    y, ht = ops.selective_scan_autograd(*args, **kw, cu_seqlens=cu)
    assert (y[:, 70:] == 0).all()
    (y.float().sum() + ht.sum()).backward()
    for t in leaves:
        assert torch.isfinite(t.grad).all()
    for t in (args[0], args[1], args[3], args[4]):
        assert (t.grad[:, 70:] == 0).all() and (t.grad[:, :70] != 0).any()
    x = torch.randn(1, 50, 24, device="cuda").requires_grad_(True)
    w = torch.randn(24, 4, device="cuda").requires_grad_(True)
    cu = torch.tensor([0, 20, 31], dtype=torch.int32, device="cuda")
    y, _ = ops.short_conv_autograd(x, w, cu_seqlens=cu)
    assert (y[:, 31:] == 0).all()
    y.sum().backward()
    assert (x.grad[:, 31:] == 0).all() and torch.isfinite(x.grad).all() and torch.isfinite(w.grad).all()


def test_second_derivatives_and_workspaces_are_refused():
    from chunkwise_delta_rule_chunk_amd import ops
    args, kw, dy, dht = _inputs(1, 70, 2, 1, 32, 32, "bf16", "fp32", 5, 1)
    x = args[0].requires_grad_(True)
    y, _ = ops.selective_scan_autograd(x, *args[1:], **kw)
    g, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().sum().backward()
    ctx = ops.selective_scan(*(t.detach() for t in args), **kw)[2]
    with pytest.raises(ValueError, match="ws must be"):
        ops.selective_scan_backward(ctx, dy, dht, ws=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws must be"):
        ops.selective_scan(*(t.detach() for t in args), **kw, ws=torch.empty(1 << 24, device="cuda"))
    from chunkwise_delta_rule_chunk_amd.binding import RewyError
    with pytest.raises(RewyError, match="workspace"):
        ops.selective_scan(*(t.detach() for t in args), **kw, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
