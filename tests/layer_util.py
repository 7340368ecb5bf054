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
