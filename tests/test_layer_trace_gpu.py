"""The trace names every kernel of a call of the operators around the token mixer, each with its
own time and launches."""
import pytest
import torch

from parity_util import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def _traced(fn, stage=None):
    from chunkwise_delta_rule_chunk_amd import binding as B
    fn()
    torch.cuda.synchronize()
    B.rewy_trace_select(stage)
    B.rewy_trace_begin()
    fn()
    fn()
    out = B.rewy_trace_end()
    B.rewy_trace_select(None)
    # the kernel's template name, in a demangled or mangled symbol
    names = ("k_norm_fwd", "k_norm_bwd", "k_colsum", "k_conv_fwd", "k_conv_bwd", "k_conv_step", "k_conv_reduce", "k_ssm_prep",
             "k_ssm_state", "k_ssm_pass", "k_ssm_fwd", "k_ssm_walk", "k_ssm_chunk", "k_ssm_gate", "k_ssm_params",
             "k_ssm_recurrent", "k_state_through")
    res = {}
    for sym, ms, n in out:
        found = [k for k in names if k in sym]
        assert len(found) == 1, sym
        res[found[0]] = res.get(found[0], 0) + n
        assert ms > 0
    return res


def test_kernels_of_each_call():
    from chunkwise_delta_rule_chunk_amd import ops
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w = rn(40, 64), rn(64)
    c = ops.rms_norm(x, w)[4]
    assert _traced(lambda: ops.rms_norm(x, w)) == dict(k_norm_fwd=2)
    assert _traced(lambda: ops.rms_norm_backward(c, x)) == dict(k_norm_bwd=2, k_colsum=2)
    cx, cw, ch = rn(1, 40, 64), rn(64, 4), rn(1, 3, 64)
    c = ops.short_conv(cx, cw)[2]
    assert _traced(lambda: ops.short_conv(cx, cw)) == dict(k_conv_fwd=2)
    assert _traced(lambda: ops.short_conv_step(cx[:, 0], ch, cw)) == dict(k_conv_step=2)
    assert _traced(lambda: ops.short_conv_backward(c, cx)) == dict(k_conv_bwd=2, k_conv_reduce=2)
    assert _traced(lambda: ops.short_conv_backward(c, cx), "k_conv_bwd") == dict(k_conv_bwd=2)
    a = (rn(1, 600, 2, 32), rn(1, 600, 2), rn(2), rn(1, 600, 1, 32), rn(1, 600, 1, 32))
    c = ops.selective_scan(*a)[2]
    assert _traced(lambda: ops.selective_scan(*a)) == dict(k_ssm_prep=2, k_ssm_state=2, k_ssm_pass=2, k_ssm_fwd=2)
    assert _traced(lambda: ops.selective_scan_recurrent(*a)) == dict(k_ssm_recurrent=2)
    assert _traced(lambda: ops.selective_scan_backward(c, a[0])) == dict(
        k_ssm_prep=2, k_ssm_state=2, k_ssm_pass=2, k_ssm_walk=2, k_ssm_chunk=2, k_ssm_gate=2, k_ssm_params=2)
    e = tuple(t[:, :0].contiguous() if t.dim() > 1 else t for t in a)
    assert _traced(lambda: ops.selective_scan(*e)) == dict(k_state_through=2)
