"""The e4m3 product has no gradient: every input that requires one is refused while
gradients are recorded, codes made by a cast among them (no GPU needed)."""
import pytest
import torch

from chunkwise_delta_rule_chunk_amd import ops

F8 = torch.float8_e4m3fn


def _args(**grad):
    a, w = torch.ones(5, 256, requires_grad=grad.get("a", False)).to(F8), torch.ones(200, 256, requires_grad=grad.get("w", False)).to(F8)
    sa, sw, b = torch.ones(5, 2), torch.ones(2, 2), torch.zeros(200)
    for name, t in (("a_scale", sa), ("w_scale", sw), ("bias", b)):
        t.requires_grad_(grad.get(name, False))
    return a, sa, w, sw, b


@pytest.mark.parametrize("name", ["a", "w", "a_scale", "w_scale", "bias"])
def test_an_input_that_requires_a_gradient_is_refused(name):
    with pytest.raises(ValueError, match="no gradient"):
        ops.e4m3_linear(*_args(**{name: True}))
    # not recorded, or detached: as far as the check of the device
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ops.e4m3_linear(*_args(**{name: True}))
    with pytest.raises(ValueError, match="GPU"):
        ops.e4m3_linear(*(t.detach() for t in _args(**{name: True})))


def test_a_leaf_of_codes_is_refused():
    a, sa, w, sw, b = _args()
    with pytest.raises(ValueError, match="no gradient"):
        ops.e4m3_linear(a, sa, torch.nn.Parameter(w), sw, b)
