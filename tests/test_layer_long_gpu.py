"""Tensors of the operators around the token mixer whose offsets pass 32 bits, and
autograd where one of two outputs is used: bit by bit what the plain call gives."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]

ROWS, STRIDE = 600, 1 << 22  # 2.5e9 elements between the first and the last row


@pytest.fixture(scope="module")
def far():
    """Rows of 4 M elements of bf16 (5 GB), of which the tests use the ends."""
    return torch.empty(ROWS, STRIDE, dtype=torch.bfloat16, device="cuda")


def _put(far, col, t):
    """t [1, ROWS, ...] in the columns col .. of the far rows"""
    n = t[0, 0].numel()
    v = far[:, col:col + n]
    v.copy_(t.reshape(ROWS, n))
    return v.unflatten(-1, t.shape[2:]).unsqueeze(0)


def test_norm(far):
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dy = (torch.randn(1, ROWS, 1000, generator=g, device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(1000, generator=g, device="cuda")
    y, s, q, sc, ctx = ops.rms_norm(x[0], w, r[0], quant="e4m3", group=128)
    xf, rf = _put(far, 0, x)[0], _put(far, STRIDE - 1000, r)[0]
    y2, s2, q2, sc2, _ = ops.rms_norm(xf, w, rf, quant="e4m3", group=128)
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(sc, sc2)
    a = ops.rms_norm_backward(ctx, dy[0])
    b = ops.rms_norm_backward(dict(ctx, s=_put(far, 0, s[None])[0]), _put(far, 3001, dy)[0])
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])


def test_convolution(far):
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(1, ROWS, 520, generator=g, device="cuda").bfloat16() for _ in range(2))
    w, h0 = torch.randn(520, 4, generator=g, device="cuda"), torch.randn(1, 3, 520, generator=g, device="cuda").bfloat16()
    y, ht, ctx = ops.short_conv(x, w, h0=h0, output_final_state=True)
    y2, ht2, ctx2 = ops.short_conv(_put(far, STRIDE - 521, x), w, h0=h0, output_final_state=True)
    assert torch.equal(y, y2) and torch.equal(ht, ht2)
    a, b = ops.short_conv_backward(ctx, dy), ops.short_conv_backward(ctx2, _put(far, 1, dy))
    for k in ("dx", "dweight", "dh0"):
        assert torch.equal(a[k], b[k]), k


def test_scan(far):
    from chunkwise_delta_rule_chunk_amd import ops
    H, V, K = 4, 64, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, b, c, dy = (rn(1, ROWS, n, v).bfloat16() for n, v in ((H, V), (1, K), (1, K), (H, V)))
    dt, al, h0 = rn(1, ROWS, H) - 3, rn(H), rn(1, H, K, V)
    y, ht, ctx = ops.selective_scan(x, dt, al, b, c, h0=h0)
    xf, bf, cf, dyf = (_put(far, col, t) for col, t in ((STRIDE - H * V, x), (8, b), (4096, c), (8192, dy)))
    y2, ht2, ctx2 = ops.selective_scan(xf, dt, al, bf, cf, h0=h0)
    assert torch.equal(y, y2) and torch.equal(ht, ht2)
    a = ops.selective_scan_backward(ctx, dy)
    out = tuple(_put(far, col, torch.zeros_like(t)) for col, t in ((1 << 20, x), (1 << 21, b), (3 << 20, c)))
    f = ops.selective_scan_backward(ctx2, dyf, out=out)
    for k in ("dx", "db", "dc", "ddt", "da_log", "dh0"):
        assert torch.equal(a[k], f[k]), k
    yr, hr = ops.selective_scan_recurrent(x, dt, al, b, c, h0=h0)
    yr2, hr2 = ops.selective_scan_recurrent(xf, dt, al, bf, cf, h0=h0)
    assert torch.equal(yr, yr2) and torch.equal(hr, hr2)


def test_one_of_two_outputs():
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(4)
    leaf = lambda *s: torch.randn(*s, generator=g, device="cuda").requires_grad_(True)  # noqa: E731
    x, r, w = leaf(5, 70), leaf(5, 70), leaf(70)
    y, s = ops.rms_norm_autograd(x, w, r)
    assert torch.equal(torch.autograd.grad(s.sum(), x)[0], torch.ones_like(x))
    y, s = ops.rms_norm_autograd(x, w, r)
    gy = torch.autograd.grad(y.square().sum(), r)[0]
    y, s = ops.rms_norm_autograd(x, w, r)
    both = torch.autograd.grad(y.square().sum() + s.sum(), r)[0]
    assert ((both - gy) - 1).abs().max() <= 2.0 ** -22 * (1 + gy.abs().max())
    x, w, h0 = leaf(1, 9, 6), leaf(6, 4), leaf(1, 3, 6)
    _, ht = ops.short_conv_autograd(x, w, h0=h0)
    gx, gw, gh = torch.autograd.grad(ht.sum(), (x, w, h0))
    want = torch.zeros_like(x)
    want[:, -3:] = 1
    assert torch.equal(gx, want) and (gw == 0).all() and (gh == 0).all()
    args = (leaf(1, 70, 2, 32), leaf(1, 70, 2), leaf(2), leaf(1, 70, 1, 32), leaf(1, 70, 1, 32))
    _, ht = ops.selective_scan_autograd(*args)
    some = torch.autograd.grad(ht.sum(), args)
    y, ht = ops.selective_scan_autograd(*args)
    full = torch.autograd.grad((y * 0).sum() + ht.sum(), args)
    for a, b in zip(some, full):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Forward and backward of the three on two streams that overlap: each as alone."""
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    sets = []
    for T in (700, 1300):
        x, r, w = rn(T, 512).bfloat16(), rn(T, 512).bfloat16(), rn(512)
        cw = rn(512, 4)
        scan = (rn(1, T, 4, 64).bfloat16(), rn(1, T, 4) - 3, rn(4), rn(1, T, 1, 128).bfloat16(), rn(1, T, 1, 128).bfloat16())
        sets.append((x, r, w, cw, scan))

    def run(x, r, w, cw, scan, stream=None):
        y, s, _, _, nc = ops.rms_norm(x, w, r, stream=stream)
        n = ops.rms_norm_backward(nc, r, stream=stream)
        z, _, cc = ops.short_conv(x[None], cw, stream=stream)
        c = ops.short_conv_backward(cc, r[None], stream=stream)
        o, ht, sc = ops.selective_scan(*scan, stream=stream)
        b = ops.selective_scan_backward(sc, scan[0], stream=stream)
        return [y, s, n["dx"], n["dweight"], z, c["dx"], c["dweight"], o, ht] + [b[k] for k in ("dx", "ddt", "da_log", "db", "dc")]

    alone = [run(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[run(*a, stream=s) for a, s in zip(sets, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(alone, pair):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
