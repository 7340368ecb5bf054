"""Calls of the operators around the token mixer that their documentation allows, bit by bit
against the plain call: captured graphs whose offsets change between replays, two graphs in
turn, every second token, single tokens cut out of longer rows, a graph of autograd used
twice, the norm's two outputs without a residual, more than two leading dimensions."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def _same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


OFFSETS = [[0, 100, 700, 900], [0, 0, 0, 900], [0, 1, 64, 65], [0, 449, 449, 890], [0, 0, 0, 0], [0, 100, 700, 900]]


def test_a_captured_call_follows_new_offsets():
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(1)
    T, H, V, G, K = 900, 4, 32, 2, 64
    x, w, ch = rn(1, T, 96).bfloat16(), rn(96, 4), rn(3, 3, 96).bfloat16()
    dy = rn(1, T, 96).bfloat16()
    a = (rn(1, T, H, V).bfloat16(), rn(1, T, H) - 3, rn(H), rn(1, T, G, K).bfloat16(), rn(1, T, G, K).bfloat16())
    h0, sdy, dht = rn(3, H, K, V), rn(1, T, H, V).bfloat16(), rn(3, H, K, V)
    cu = torch.tensor(OFFSETS[0], dtype=torch.int32, device="cuda")

    def run():
        y, ht, c = ops.short_conv(x, w, h0=ch, cu_seqlens=cu, output_final_state=True, clear=True)
        gc = ops.short_conv_backward(c, dy, ch, clear=True)
        o, st, s = ops.selective_scan(*a, h0=h0, cu_seqlens=cu, clear=True)
        gs = ops.selective_scan_backward(s, sdy, dht, clear=True)
        return [y, ht, *gc.values(), o, st, *gs.values()]

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
        assert all(torch.isfinite(t.float()).all() for t in want if t is not None)


def test_two_graphs_in_turn():
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(2)
    sets = [(rn(1, T, 4, 64).bfloat16(), rn(1, T, 4) - 3, rn(4), rn(1, T, 1, 64).bfloat16(), rn(1, T, 1, 64).bfloat16())
            for T in (700, 1300)]

    def run(a):
        y, ht, c = ops.selective_scan(*a)
        g = ops.selective_scan_backward(c, a[0], ht)
        n = ops.rms_norm(y.flatten(2), quant="e4m3", group=64)
        return [y, ht, *g.values(), n[0], n[2].view(torch.uint8), n[3]]

    want = [run(a) for a in sets]
    torch.cuda.synchronize()
    graphs = []
    for a in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(a)
        graphs.append((graph, out))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert _same(out, w)


def test_spaced_tokens_and_single_ones():
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(3)
    x, w, h0 = rn(3, 20, 64).bfloat16(), rn(64, 4), rn(3, 3, 64).bfloat16()
    y, ht, c = ops.short_conv(x[:1, ::2], w, h0=h0[:1], output_final_state=True)
    y2, ht2, c2 = ops.short_conv(x[:1, ::2].contiguous(), w, h0=h0[:1], output_final_state=True)
    dy = rn(1, 10, 64).bfloat16()
    assert _same((y, ht, *ops.short_conv_backward(c, dy).values()), (y2, ht2, *ops.short_conv_backward(c2, dy).values()))
    one, st = ops.short_conv_step(x[:, 7], h0, w)
    full, ht, _ = ops.short_conv(x[:, 7:8], w, h0=h0, output_final_state=True)
    assert torch.equal(one[:, None], full) and torch.equal(st, ht)
    a = (rn(3, 20, 2, 32).bfloat16(), rn(3, 20, 2) - 3, rn(2), rn(3, 20, 1, 64).bfloat16(), rn(3, 20, 1, 64).bfloat16())
    s0 = rn(3, 2, 64, 32)
    cut = lambda t: t[:, 11:12]  # noqa: E731
    sl = (cut(a[0]), cut(a[1]).contiguous(), a[2], cut(a[3]), cut(a[4]))
    cp = tuple(t.contiguous() for t in sl)
    assert _same(ops.selective_scan_recurrent(*sl, h0=s0), ops.selective_scan_recurrent(*cp, h0=s0))
    assert _same(ops.selective_scan(*sl, h0=s0)[:2], ops.selective_scan(*cp, h0=s0)[:2])


def test_norm_shapes_and_outputs():
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(4)
    x, w = rn(2, 3, 5, 200), rn(70)
    part = x[..., 30:100]
    for q in (None, "int8"):
        a, b = (ops.rms_norm(t, w, quant=q, group=32 if q else 0) for t in (part, part.reshape(-1, 70)))
        assert a[0].shape == part.shape and torch.equal(a[0].reshape(-1, 70), b[0])
        if q:
            assert a[2].shape == part.shape and torch.equal(a[2].reshape(-1, 70), b[2]) and torch.equal(a[3], b[3])
    row, alone = ops.rms_norm(x[0, 0, 0, :70], w)[0], ops.rms_norm(x[0, 0, :1, :70], w)[0]
    assert torch.equal(row, alone[0])
    # without a residual the second output is x itself, and its adjoint joins y's
    leaf = rn(6, 70).requires_grad_(True)
    y, s = ops.rms_norm_autograd(leaf, w)
    assert torch.equal(s, leaf)
    r = rn(6, 70)
    both, = torch.autograd.grad((y * r).sum() + (s * 3).sum(), leaf)
    gy, = torch.autograd.grad((ops.rms_norm_autograd(leaf, w)[0] * r).sum(), leaf)
    assert (both - (gy + 3)).abs().max() <= 2.0 ** -22 * (4 + gy.abs().max())
    only, = torch.autograd.grad((ops.rms_norm_autograd(leaf, w)[1] * 3).sum(), leaf)
    assert torch.equal(only, torch.full_like(leaf, 3.0))


def test_a_graph_of_autograd_used_twice():
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(5)
    lf = lambda *s: rn(*s).requires_grad_(True)  # noqa: E731
    a = (lf(1, 90, 2, 32), lf(1, 90, 2), lf(2), lf(1, 90, 1, 32), lf(1, 90, 1, 32))
    x, w, n = lf(1, 90, 64), lf(64, 3), lf(64)
    u, _ = ops.short_conv_autograd(x, w, cu_seqlens=[0, 30, 90])
    y, _ = ops.selective_scan_autograd(u.unflatten(-1, (2, 32)), *a[1:], cu_seqlens=[0, 30, 90])
    z, _ = ops.rms_norm_autograd(y.flatten(2), n, u)
    leaves = (x, w, n, *a[1:])
    once = torch.autograd.grad(z.sum(), leaves, retain_graph=True)
    again = torch.autograd.grad(z.sum(), leaves)
    assert _same(once, again)


def test_states_and_their_adjoints_left_out():
    """No initial state is a state of zeros, no adjoint one of zeros; dh0 may be asked for without h0."""
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(6)
    for T, dt in ((600, torch.bfloat16), (70, torch.float32)):
        a = (rn(2, T, 2, 64).to(dt), rn(2, T, 2) - 3, rn(2), rn(2, T, 1, 32).to(dt), rn(2, T, 1, 32).to(dt))
        z, dy = torch.zeros(2, 2, 32, 64, device="cuda"), rn(2, T, 2, 64).to(dt)
        y, ht, c = ops.selective_scan(*a)
        y0, ht0, c0 = ops.selective_scan(*a, h0=z)
        assert torch.equal(y, y0) and torch.equal(ht, ht0)
        g, g0 = ops.selective_scan_backward(c, dy, want_dh0=True), ops.selective_scan_backward(c0, dy, z)
        for k in ("dx", "db", "dc", "dh0"):
            assert torch.equal(g[k], g0[k]), k
        for k in ("ddt", "da_log"):  # (a state that is given ends the decay gradient's chains elsewhere)
            assert (g[k].double() - g0[k].double()).norm() <= 1e-5 * g0[k].double().norm(), k
        assert ops.selective_scan_backward(c0, dy, z, want_dh0=False)["dh0"] is None
    x, w, dy = rn(2, 50, 36), rn(36, 4), rn(2, 50, 36)
    z = torch.zeros(2, 3, 36, device="cuda")
    y, ht, c = ops.short_conv(x, w, output_final_state=True)
    y0, ht0, c0 = ops.short_conv(x, w, h0=z, output_final_state=True)
    assert torch.equal(y, y0) and torch.equal(ht, ht0)
    g, g0 = ops.short_conv_backward(c, dy), ops.short_conv_backward(c0, dy, z)
    assert torch.equal(g["dx"], g0["dx"]) and torch.equal(g["dweight"], g0["dweight"]) and g["dh0"] is None


def test_two_threads_at_once():
    """Each thread on a stream of its own; errors of one are not the other's."""
    import threading

    from chunkwise_delta_rule_chunk_amd import binding as B
    from chunkwise_delta_rule_chunk_amd import ops
    rn = _gen(7)
    sets = [(rn(1, T, 4, 64).bfloat16(), rn(1, T, 4) - 3, rn(4), rn(1, T, 1, 64).bfloat16(), rn(1, T, 1, 64).bfloat16())
            for T in (500, 900)]

    def once(a):
        y, ht, c = ops.selective_scan(*a)
        return [y, ht, *ops.selective_scan_backward(c, a[0], ht).values()]

    want = [once(a) for a in sets]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    out = once(sets[i])
                    s.synchronize()
                    assert _same(out, want[i])
                    with pytest.raises(B.RewyError, match="bad eps"):
                        ops.rms_norm(sets[i][0], eps=-1.0)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
