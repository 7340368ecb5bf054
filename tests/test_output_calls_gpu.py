"""Calls of the attention with a constant decay, the group norm and the e4m3 product that
their documentation allows: other streams and threads, captured graphs whose offsets change
between replays, padded batches, infinities, updates in place, slices as outputs, long
sequences, offsets past 32 bits, differences, the trace.  Unless a bound is stated, bit by
bit what the plain call gives."""
import threading

import pytest
import torch

from layer_util import U32, close
from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

F8 = torch.float8_e4m3fn


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def _same(a, b):
    raw = lambda t: t.view(torch.uint8) if t.dtype == F8 else t  # noqa: E731
    return all((p is None and q is None) or torch.equal(raw(p), raw(q)) for p, q in zip(a, b, strict=True))


def _attn(rn, T, H, G, K, V, dt=torch.bfloat16, B=1):
    return rn(B, T, H, K).to(dt), rn(B, T, G, K).to(dt), rn(B, T, G, V).to(dt), -torch.linspace(0.004, 0.6, H, device="cuda")


def _everything(rn, T=700):
    """One call of each operator; returns the call."""
    a = _attn(rn, T, 4, 2, 64, 64)
    h0, do, dht = rn(1, 4, 64, 64), rn(1, T, 4, 64).bfloat16(), rn(1, 4, 64, 64)
    gate, w, b = rn(1, T, 256).bfloat16(), rn(256), rn(256)
    wq, sw = rn(130, 256).mul(30).to(F8), rn(2, 2).exp()

    def run():
        o, ht, c = ops().decay_attention(*a, h0=h0)
        gr = ops().decay_attention_backward(c, do, dht)
        s = ops().decay_attention_recurrent(*(t[:, :3] for t in a[:3]), a[3], h0=h0)
        y, q, sc, n = ops().group_norm(o.flatten(2), w, b, gate, groups=4, quant="e4m3", group=128)
        gn = ops().group_norm_backward(n, do.flatten(2))
        odd = ops().group_norm(o.flatten(2)[..., :253], groups=11, quant="int8")
        go = ops().group_norm_backward(odd[3], do.flatten(2)[..., :253])
        z = ops().e4m3_linear(q, sc, wq, sw)
        z2 = ops().e4m3_linear(q[:, :9], sc[:9], wq, sw, dtype=torch.float32)
        return [o, ht, *gr.values(), *s, y, q, sc, *gn.values(), *odd[:3], *go.values(), z, z2]
    return run


def ops():
    from chunkwise_delta_rule_chunk_amd import ops as o
    return o


def test_another_stream_and_two_threads():
    runs = [_everything(_gen(s), T) for s, T in ((1, 700), (2, 391))]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = runs[0]()
    st.synchronize()
    assert _same(want[0], got)
    outs, fails = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    outs[i] = runs[i]()
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            fails.append(e)
    th = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in th:
        t.start()
    for t in th:
        t.join()
    assert not fails and all(_same(w, o) for w, o in zip(want, outs))


def test_the_stream_argument():
    rn = _gen(3)
    a, x = _attn(rn, 300, 2, 1, 64, 32), rn(300, 64)
    wq, sw = rn(70, 64).mul(30).to(F8), rn(1, 1).exp()
    st = torch.cuda.Stream()

    def run(stream):
        o, ht, c = ops().decay_attention(*a, stream=stream)
        g = ops().decay_attention_backward(c, o, stream=stream)
        s = ops().decay_attention_recurrent(*a, stream=stream)
        y, q, sc, n = ops().group_norm(x, groups=4, quant="e4m3", stream=stream)
        gn = ops().group_norm_backward(n, y, stream=stream)
        return [o, ht, *g.values(), *s, y, q, sc, *gn.values(), ops().e4m3_linear(q, sc, wq, sw, stream=stream)]

    want = run(None)
    st.wait_stream(torch.cuda.current_stream())
    got = run(st)
    st.synchronize()
    assert _same(want, got)


def test_two_graphs_in_turn():
    runs = [_everything(_gen(s), T) for s, T in ((4, 900), (5, 130))]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    graphs = []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = r()
        graphs.append((graph, out))
    for _ in range(3):
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(_same(out, w) for (_, out), w in zip(graphs, want))
        runs[0]()  # the program's own work in between


OFFSETS = [[0, 100, 700, 900], [0, 0, 0, 900], [0, 1, 64, 65], [0, 449, 449, 890], [0, 0, 0, 0], [0, 100, 700, 900]]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_captured_call_follows_new_offsets(dt):
    rn = _gen(6)
    T, H, G, K, V = 900, 4, 2, 64, 32
    a = _attn(rn, T, H, G, K, V, dt)
    h0, do, dht = rn(3, H, K, V), rn(1, T, H, V).to(dt), rn(3, H, K, V)
    cu = torch.tensor(OFFSETS[0], dtype=torch.int32, device="cuda")

    def run():
        o, ht, c = ops().decay_attention(*a, h0=h0, cu_seqlens=cu, clear=True)
        g = ops().decay_attention_backward(c, do, dht, clear=True)
        return [o, ht, *g.values()]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for off in OFFSETS:
        cu.copy_(torch.tensor(off, dtype=torch.int32))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(want, out), off
        # each sequence as a call of its own: the segments' borders differ, so bounds (half a
        # step of 16 bits on each side and its operands' roundings, as in the attention's own test)
        for n in range(3):
            t0, t1 = off[n], off[n + 1]
            if t1 == t0:
                assert torch.equal(out[1][n], h0[n])
                continue
            cut = lambda t: t[:, t0:t1].contiguous()  # noqa: E731
            o, ht, c = ops().decay_attention(*map(cut, a[:3]), a[3], h0=h0[n:n + 1])
            g = ops().decay_attention_backward(c, cut(do), dht[n:n + 1])
            bound = 4 * 2.0 ** -8 if dt == torch.bfloat16 else 2e-5
            for x, y in zip((o, g["dq"], g["dk"], g["dv"]), (out[0], *out[2:5])):
                assert (x.double() - cut(y).double()).norm() <= bound * x.double().norm()
            assert (ht[0] - out[1][n]).double().norm() <= 2e-5 * ht.double().norm()
            assert (g["dh0"][0] - out[5][n]).double().norm() <= 2e-5 * g["dh0"].double().norm()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_behind_the_last_sequence(dt):
    """Neither read (they hold NaN) nor written, or cleared where that is asked for; offsets past the end
    and decreasing ones are held to the packed axis."""
    rn = _gen(7)
    T, H, G, K, V, end = 500, 4, 2, 64, 64, 333
    a = _attn(rn, T, H, G, K, V, dt)
    do = rn(1, T, H, V).to(dt)
    cu = torch.tensor([0, 200, end], dtype=torch.int32, device="cuda")
    cut = lambda t: t[:, :end].contiguous()  # noqa: E731
    o1, ht1, c1 = ops().decay_attention(*map(cut, a[:3]), a[3], cu_seqlens=cu)
    g1 = ops().decay_attention_backward(c1, cut(do))
    s1 = ops().decay_attention_recurrent(*map(cut, a[:3]), a[3], cu_seqlens=cu)
    for t in (*a[:3], do):
        t[:, end:] = float("nan")
    o, ht, c = ops().decay_attention(*a, cu_seqlens=cu, clear=True)
    g = ops().decay_attention_backward(c, do, clear=True)
    s = ops().decay_attention_recurrent(*a, cu_seqlens=cu)
    # (segments are as long as the packed axis asks for, so only the token-serial form is bit by bit)
    assert torch.equal(cut(s[0]), s1[0]) and torch.equal(s[1], s1[1])
    bound = 4 * 2.0 ** -8 if dt == torch.bfloat16 else 2e-5
    for x, y in ((o, o1), (g["dq"], g1["dq"]), (g["dk"], g1["dk"]), (g["dv"], g1["dv"])):
        assert (cut(x).double() - y.double()).norm() <= bound * y.double().norm()
        assert not x[:, end:].any()
    assert (ht - ht1).double().norm() <= 2e-5 * ht1.double().norm()
    mark = [torch.full_like(t, 7.0) for t in a[:3]]
    ops().decay_attention_backward(c, do, out=mark)
    assert _same([cut(t) for t in mark], [cut(g[n]) for n in ("dq", "dk", "dv")])
    assert all((t[:, end:] == 7).all() for t in mark)
    for t in (*a[:3], do):
        t[:, end:] = 0.25
    for off, plain in (([0, 400, 900], [0, 400, T]), ([0, 300, 100], [0, 300, 300]), ([0, -5, T], [0, 0, T])):
        p, r = (ops().decay_attention(*a, cu_seqlens=torch.tensor(t, dtype=torch.int32, device="cuda"), clear=True)
                for t in (off, plain))
        if off[2] > off[1]:
            assert _same(p[:2], r[:2])
        else:  # the last offset is what rows behind it go by: the first sequence is still whole
            assert torch.equal(p[1], r[1])


@pytest.mark.parametrize("dt,bad", [(torch.bfloat16, float("nan")), (torch.bfloat16, float("inf")), (torch.float32, float("-inf"))])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_an_infinity_reaches_its_token_and_the_ones_behind(dt, bad, which):
    rn = _gen(8)
    H, G, K, V, lens, at = 4, 2, 64, 32, [150, 300, 90], 150 + 100
    T = sum(lens)
    a = list(_attn(rn, T, H, G, K, V, dt))
    cu = torch.tensor([0, 150, 450, 540], dtype=torch.int32, device="cuda")
    o1, ht1, _ = ops().decay_attention(*a, cu_seqlens=cu)
    s1, _ = ops().decay_attention_recurrent(*a, cu_seqlens=cu)
    a[which] = a[which].clone()
    a[which][0, at, 1, 3] = bad
    o, ht, _ = ops().decay_attention(*a, cu_seqlens=cu)
    s, st = ops().decay_attention_recurrent(*a, cu_seqlens=cu)
    heads = [1] if which == 0 else [2, 3]
    for got, plain in ((o, o1), (s, s1)):
        clean = torch.ones(T, H, dtype=torch.bool, device="cuda")
        clean[at:at + 1 if which == 0 else 450, heads] = False
        assert torch.equal(got[0][clean], plain[0][clean])
        # (a value's infinity is in its own column only)
        assert not torch.isfinite(got[0, at, heads]).all(-1).any()
    if which:
        for fin in (ht, st):
            assert not torch.isfinite(fin[1, heads]).flatten(1).all(1).any()
            assert torch.isfinite(fin[[0, 2]]).all() and torch.isfinite(fin[1, :2]).all()
    else:
        assert torch.equal(ht, ht1)


def test_updates_in_place_and_slices_as_outputs():
    rn = _gen(9)
    a, h0 = _attn(rn, 5, 8, 8, 128, 128, B=3), rn(3, 8, 128, 128)
    o, ht = ops().decay_attention_recurrent(*a, h0=h0)
    state = h0.clone()
    for t in range(5):
        ot, same = ops().decay_attention_recurrent(*(x[:, t:t + 1] for x in a[:3]), a[3], h0=state, ht=state)
        assert same is state and torch.equal(ot[:, 0], o[:, t])
    assert torch.equal(state, ht)
    # gradients straight into the joint projection's row, from a row of adjoints that is a slice
    H, G, K, V, T = 4, 2, 64, 32, 300
    row = rn(2, T, H * K + G * (K + V) + 64).bfloat16()
    cut = lambda r: [t.unflatten(-1, (n, -1)) for t, n in zip(r[..., :-64].split([H * K, G * K, G * V], -1), (H, G, G))]  # noqa: E731
    q, k, v = cut(row)
    g = -torch.rand(H, device="cuda")
    o, _, c = ops().decay_attention(q, k, v, g)
    wide = rn(2, T, H * V + 32).bfloat16()
    do = wide[..., 16:-16].unflatten(-1, (H, V))
    want = ops().decay_attention_backward(c, do.contiguous())
    drow = torch.full_like(row, 7.0)
    ops().decay_attention_backward(c, do, out=cut(drow))
    assert _same(cut(drow), [want[n] for n in ("dq", "dk", "dv")]) and (drow[..., -64:] == 7).all()


@pytest.mark.parametrize("packed", [None, "list", "device"])
def test_autograd(packed):
    """The wrappers' gradients are the explicit calls'; saved tensors may be kept on the host; a
    graph may be walked twice and gradients of broadcast or shared inputs join; no second derivative."""
    rn = _gen(10)
    T, H, G, K, V = 150, 4, 2, 64, 32
    row = rn(1, T, 704).bfloat16().requires_grad_(True)
    h0, nw = rn(1 if packed is None else 2, H, K, V).requires_grad_(True), rn(H * V).requires_grad_(True)
    g, r = -torch.rand(H, device="cuda"), rn(1, T, H * V).bfloat16()
    cu = None if packed is None else [0, 70, T]
    if packed == "device":
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def parts():
        q, k, v = row[..., :448].split([H * K, G * K, G * V], -1)
        return q.unflatten(-1, (H, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (G, V)), row[..., 500:500 + H * V]

    def loss():
        q, k, v, gate = parts()
        o, ht = ops().decay_attention_autograd(q, k, v, g, h0=h0, cu_seqlens=cu)
        y = ops().group_norm_autograd(o.flatten(2), nw, None, gate, groups=H)
        return (y * r).float().sum() + ht.sum()

    leaves = (row, h0, nw)
    out = loss()
    want = torch.autograd.grad(out, leaves, retain_graph=True)
    assert _same(want, torch.autograd.grad(out, leaves))
    with torch.autograd.graph.save_on_cpu():
        out = loss()
    assert _same(want, torch.autograd.grad(out, leaves))
    with torch.no_grad():
        q, k, v, gate = parts()
        o, ht, c = ops().decay_attention(q, k, v, g, h0=h0, cu_seqlens=cu)
        _, _, _, n = ops().group_norm(o.flatten(2), nw, None, gate, groups=H)
        gn = ops().group_norm_backward(n, r)
        ga = ops().decay_attention_backward(c, gn["dx"].view_as(o), torch.ones_like(ht))
        drow = torch.zeros_like(row)
        drow[..., :448] = torch.cat([ga[t].flatten(2) for t in ("dq", "dk", "dv")], -1)
        drow[..., 500:500 + H * V] = gn["dgate"]
    assert _same(want, (drow, ga["dh0"], gn["dweight"]))
    # one tensor as two arguments, and a row used by every token
    x, one = rn(1, T, 2, 64).requires_grad_(True), rn(1, 1, 2, 64).requires_grad_(True)
    o, _ = ops().decay_attention_autograd(x, x, one.expand(1, T, 2, 64).contiguous(), g[:2])
    gx, g1 = torch.autograd.grad(o.sum(), (x, one), create_graph=True)
    _, _, c = ops().decay_attention(x, x, one.expand(1, T, 2, 64).contiguous(), g[:2])
    e = ops().decay_attention_backward(c, torch.ones_like(o))
    assert torch.equal(gx, e["dq"] + e["dk"])
    assert (g1 - e["dv"].sum(1, keepdim=True)).abs().max() <= 2 * T * U32 * e["dv"].abs().sum(1).max()
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        gx.sum().backward()
    only, = torch.autograd.grad(ops().decay_attention_autograd(x, x.detach(), x.detach(), g[:2])[1].sum(), x, allow_unused=True)
    assert only is None or not only.any()  # the state does not depend on the queries
    if packed == "device":
        o, _ = ops().decay_attention_autograd(*parts()[:3], g, h0=h0, cu_seqlens=cu)
        cu[1] += 5
        with pytest.raises(RuntimeError, match="inplace operation"):
            o.sum().backward()


def test_gradients_are_differences():
    """The attention is linear in each of q, k, v and the state, so a difference over any step is the
    gradient's product with it.  Each of the three sums is off by at most (300 + 4 chunks) U of the
    sum of its terms' magnitudes (the attention's own test), and each magnitude is at most that of
    the call with |input| + |step|, which the call itself gives within that bound again."""
    rn = _gen(11)
    T, H, G, K, V = 400, 4, 2, 32, 64
    a, h0 = _attn(rn, T, H, G, K, V, torch.float32), rn(1, H, K, V)
    do, dht = rn(1, T, H, V), rn(1, H, K, V)

    def loss(q, k, v, g, h, w=do, wh=dht):
        o, ht, c = ops().decay_attention(q, k, v, g, h0=h)
        return (o.double() * w.double()).sum() + (ht.double() * wh.double()).sum(), c
    _, c = loss(*a, h0)
    g = ops().decay_attention_backward(c, do, dht)
    ins = [*a[:3], h0]
    for i, n in enumerate(("dq", "dk", "dv", "dh0")):
        d = rn(*ins[i].shape)
        moved = [t + d if j == i else t for j, t in enumerate(ins)]
        # (the step as it was taken, the sum's rounding with it)
        step = moved[i].double() - ins[i].double()
        diff = loss(*moved[:3], a[3], moved[3])[0] - loss(*a, h0)[0]
        m = [t.abs() + (d.abs() if j == i else 0) for j, t in enumerate(ins)]
        mag = loss(*m[:3], a[3], m[3], do.abs(), dht.abs())[0]
        bound = (300 + 4 * 7 + 2) * U32
        assert abs(diff - (g[n].double() * step).sum()) <= 3.01 * bound * mag, n


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_long_sequence(dt):
    """Against the token-serial form, whose state takes three roundings a token; magnitudes
    from the same form on absolute values (itself within 1 + 1e-2)."""
    rn = _gen(12)
    T, H, K, V = 40000, 2, 32, 64
    a, h0 = _attn(rn, T, H, 1, K, V, dt), rn(1, H, K, V)
    a = (*a[:3], torch.tensor([-1e-5, -0.3], device="cuda"))
    o, ht, _ = ops().decay_attention(*a, h0=h0)
    wide = [t.float() for t in a]
    s, st = ops().decay_attention_recurrent(*wide, h0=h0)
    m, mt = ops().decay_attention_recurrent(*(t.abs() for t in wide[:3]), a[3], h0=h0.abs())
    fp = 1.01 * (600 + 4 * T + T / 16) * U32
    op = 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -16 if dt == torch.bfloat16 else 0
    close(o, s, (fp + op) * m, "o")
    close(ht, st, fp * mt, "ht")


ROWS, STRIDE = 600, 1 << 22  # 2.5e9 elements between the first and the last row


def test_rows_far_apart():
    far = torch.empty(ROWS, STRIDE, dtype=torch.bfloat16, device="cuda")
    rn = _gen(13)

    def put(col, t):
        n = t[0, 0].numel()
        v = far[:, col:col + n]
        v.copy_(t.reshape(ROWS, n))
        return v.unflatten(-1, t.shape[2:]).unsqueeze(0)

    H, G, K, V = 4, 2, 64, 32
    a, do = _attn(rn, ROWS, H, G, K, V), rn(1, ROWS, H, V).bfloat16()
    o, ht, c = ops().decay_attention(*a)
    g = ops().decay_attention_backward(c, do)
    s = ops().decay_attention_recurrent(*a)
    fa = (put(0, a[0]), put(STRIDE - 512, a[1]), put(STRIDE - 256, a[2]), a[3])
    o2, ht2, c2 = ops().decay_attention(*fa)
    assert torch.equal(o, o2) and torch.equal(ht, ht2)
    out = [put(4096 * (i + 1), torch.zeros_like(t)) for i, t in enumerate(a[:3])]
    ops().decay_attention_backward(c2, put(20480, do), out=out)
    assert _same(out, [g[n] for n in ("dq", "dk", "dv")])
    assert _same(s, ops().decay_attention_recurrent(*fa))

    for D, groups in ((1024, 8), (1010, 10)):
        x, z, dy, w = rn(ROWS, D).bfloat16(), rn(ROWS, D).bfloat16(), rn(ROWS, D).bfloat16(), rn(D)
        kw = dict(groups=groups, quant="e4m3", group=128)
        *y, c = ops().group_norm(x, w, None, z, **kw)
        fx, fz, fdy = put(0, x[None])[0], put(STRIDE - D, z[None])[0], put(2048, dy[None])[0]
        *y2, c2 = ops().group_norm(fx, w, None, fz, **kw)
        assert _same(y, y2)
        assert _same(ops().group_norm_backward(c, dy).values(), ops().group_norm_backward(c2, fdy).values())

    # rows of codes 4 MB apart, 2.4 and 5 GB in all
    codes = far.view(torch.uint8).view(-1).as_strided((2 * ROWS, STRIDE), (STRIDE, 1))
    for N in (40, 2 * ROWS):
        x, w = rn(2 * ROWS, 272).mul(40).to(F8), rn(N, 272).mul(40).to(F8)
        sx, sw = rn(2 * ROWS, 3).exp(), rn(N, 3).exp()
        fx, fw = codes[:, :272], codes[:N, STRIDE - 272:]
        fx.copy_(x.view(torch.uint8))
        fw.copy_(w.view(torch.uint8))
        for dtype in (torch.bfloat16, torch.float32):
            assert torch.equal(ops().e4m3_linear(x, sx, w, sw, dtype=dtype),
                               ops().e4m3_linear(fx.view(F8), sx, fw.view(F8), sw, dtype=dtype))
            assert torch.equal(ops().e4m3_linear(x[:30], sx[:30], w, sw, dtype=dtype),
                               ops().e4m3_linear(fx.view(F8)[:30], sx[:30], fw.view(F8), sw, dtype=dtype))


def test_a_product_of_more_than_2_31_elements():
    rn = _gen(14)
    M, N, K = 70000, 32768, 32
    a, w = rn(M, K).mul(40).to(F8), rn(N, K).mul(40).to(F8)
    sa, sw = rn(M, 1).exp(), rn(N // 128, 1).exp()
    y = ops().e4m3_linear(a, sa, w, sw)
    for m in (0, 65535, M - 300):
        # (the same kernel on part of the rows, whose tiles hold the same products)
        ref = (a[m:m + 300].double() * sa[m:m + 300].double()) @ (w.double() * sw.double().repeat_interleave(128, 0)).t()
        mag = (a[m:m + 300].double().abs() * sa[m:m + 300].double()) @ (w.double().abs() * sw.double().repeat_interleave(128, 0)).t()
        # 16-bit outputs of many rows: 2^-10 of the magnitudes and the fp32 sums (the product's own test)
        close(y[m:m + 300], ref, (134 * U32 + 2.0 ** -10) * mag, "y")


def test_long_products():
    """Many blocks of 128, each with its scales, in every kernel of the product."""
    rn = _gen(15)
    K = 8208
    w, sw = rn(300, K).mul(40).to(F8), rn(3, 65).exp()
    for M in (7, 40, 300):
        a, sa = rn(M, K).mul(40).to(F8), rn(M, 65).exp()
        wide = lambda s: s.double().repeat_interleave(128, 1)[:, :K]  # noqa: E731
        A, W = a.double() * wide(sa), w.double() * wide(sw.repeat_interleave(128, 0)[:300])
        ref, mag = A @ W.t(), A.abs() @ W.abs().t()
        for dtype in (torch.float32, torch.bfloat16):
            y = ops().e4m3_linear(a, sa, w, sw, dtype=dtype)
            exact = dtype == torch.float32 or M <= 64
            close(y, ref, ((133 + 65) * U32 + (0 if exact else 2.0 ** -10)) * mag, f"y {M}")


def test_more_rows_than_a_launch_has_along_x():
    """Rows of one vector, more than 2^20 blocks."""
    rn = _gen(16)
    M = 33_000_000
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    x[-1000:] = rn(1000, 8).bfloat16()
    y, _, _, c = ops().group_norm(x, groups=2)
    y2, _, _, c2 = ops().group_norm(x[-1000:], groups=2)
    assert torch.equal(y[-1000:], y2) and not y[:-1000].any()
    d = ops().group_norm_backward(c, x)["dx"]
    assert torch.equal(d[-1000:], ops().group_norm_backward(c2, x[-1000:])["dx"])


def test_trace_names_every_kernel():
    from chunkwise_delta_rule_chunk_amd import binding as B
    rn = _gen(17)

    def traced(fn):
        fn()
        torch.cuda.synchronize()
        B.rewy_trace_begin()
        fn()
        fn()
        names = ("k_decay_state", "k_decay_pass", "k_decay_fwd", "k_decay_bwd", "k_decay_sum", "k_decay_recurrent",
                 "k_gnorm_fwd", "k_gnorm_bwd", "k_colsum", "k_mm8_rows", "k_mm8_tile")
        res = {}
        for sym, ms, n in B.rewy_trace_end():
            found = [k for k in names if k in sym]
            assert len(found) == 1 and ms > 0, sym
            res[found[0]] = res.get(found[0], 0) + n
        return res

    a = _attn(rn, 600, 4, 2, 64, 64)
    o, _, c = ops().decay_attention(*a)
    assert traced(lambda: ops().decay_attention(*a)) == dict(k_decay_state=2, k_decay_pass=2, k_decay_fwd=2)
    assert traced(lambda: ops().decay_attention_backward(c, o)) == dict(k_decay_state=2, k_decay_pass=2, k_decay_bwd=2, k_decay_sum=2)
    short = (*(t[:, :100] for t in a[:3]), a[3])
    assert traced(lambda: ops().decay_attention(*short, output_final_state=False)) == dict(k_decay_fwd=2)
    assert traced(lambda: ops().decay_attention_recurrent(*short)) == dict(k_decay_recurrent=2)
    x, w = rn(40, 64), rn(64)
    for groups in (4, 1, 64):
        c = ops().group_norm(x, w, groups=groups)[3]
        assert traced(lambda: ops().group_norm(x, w, groups=groups)) == dict(k_gnorm_fwd=2)
        assert traced(lambda: ops().group_norm_backward(c, x)) == dict(k_gnorm_bwd=2, k_colsum=2)
    for M, name in ((5, "k_mm8_rows"), (100, "k_mm8_tile")):
        q, s, wq, sw = rn(M, 64).to(F8), rn(M, 1), rn(70, 64).to(F8), rn(1, 1)
        assert traced(lambda: ops().e4m3_linear(q, s, wq, sw)) == {name: 2}
