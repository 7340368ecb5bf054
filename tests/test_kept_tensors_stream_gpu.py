"""What a forward keeps for its backward (states, statistics, offsets of a list) belongs to
the forward's stream.  A backward on another stream marks it as used there, so that memory
that the caller lets go while that stream is still at work is not given out again."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def decay(rn):
    from chunkwise_delta_rule_chunk_amd import ops
    q = rn(1, 4096, 16, 64).bfloat16()
    g = -torch.rand(16, device="cuda")
    return (lambda **kw: ops.decay_attention(q, q, q, g, **kw)[2]), (lambda c, **kw: ops.decay_attention_backward(c, q, **kw)), ("states",)


def gnorm(rn):
    from chunkwise_delta_rule_chunk_amd import ops
    x = rn(40000, 256).bfloat16()
    return (lambda **kw: ops.group_norm(x, groups=32, **kw)[3]), (lambda c, **kw: ops.group_norm_backward(c, x, **kw)), ("mean", "rstd")


def rms(rn):
    from chunkwise_delta_rule_chunk_amd import ops
    x = rn(1 << 20, 32).bfloat16()
    return (lambda **kw: ops.rms_norm(x, **kw)[4]), (lambda c, **kw: ops.rms_norm_backward(c, x, **kw)), ("rstd",)


def offsets(n):
    return list(range(n + 1))


def conv(rn):
    from chunkwise_delta_rule_chunk_amd import ops
    x, w = rn(1, 400000, 8).bfloat16(), rn(8, 4).bfloat16()
    cu = offsets(400000)
    return (lambda **kw: ops.short_conv(x, w, cu_seqlens=cu, **kw)[2]), (lambda c, **kw: ops.short_conv_backward(c, x, **kw)), ("cu",)


def scan(rn):
    from chunkwise_delta_rule_chunk_amd import ops
    x = rn(1, 300000, 1, 32).bfloat16()
    dt, al, cu = rn(1, 300000, 1), torch.zeros(1, device="cuda"), offsets(300000)
    return ((lambda **kw: ops.selective_scan(x, dt, al, x, x, cu_seqlens=cu, output_final_state=False, **kw)[2]),
            (lambda c, **kw: ops.selective_scan_backward(c, x, **kw)), ("cu",))


@pytest.mark.parametrize("argument", [False, True])
@pytest.mark.parametrize("op", [decay, gnorm, rms, conv, scan])
def test_kept_memory_is_not_given_out_while_the_backward_runs(op, argument):
    gen = torch.Generator(device="cuda").manual_seed(1)
    fwd, bwd, names = op(lambda *s: torch.randn(*s, generator=gen, device="cuda"))
    busy = torch.randn(8192, 8192, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(fn, stream, *args):
        if argument:
            return fn(*args, stream=stream)
        with torch.cuda.stream(stream):
            return fn(*args)

    want = bwd(fwd())  # (loads the kernels)
    torch.cuda.synchronize()
    ctx = call(fwd, a)
    kept = [ctx[n] for n in names]
    assert all(t is not None and t.numel() * t.element_size() >= 1 << 20 for t in kept)
    shapes, places = [(t.numel(), t.dtype) for t in kept], {t.data_ptr() for t in kept}
    del kept
    b.wait_stream(a)
    with torch.cuda.stream(b):
        for _ in range(20):
            busy = busy @ busy * 1e-2
    got = call(bwd, b, ctx)
    del ctx
    late = torch.cuda.Event()
    late.record(b)
    with torch.cuda.stream(a):
        new = [torch.empty(n, dtype=dt, device="cuda") for n, dt in shapes for _ in range(3)]
    assert not late.query()  # (the backward is still waiting for its turn)
    assert places.isdisjoint(t.data_ptr() for t in new)
    for t in new:
        with torch.cuda.stream(a):
            t.fill_(0)
    torch.cuda.synchronize()
    assert all((want[k] is None and got[k] is None) or torch.equal(want[k], got[k]) for k in want)
