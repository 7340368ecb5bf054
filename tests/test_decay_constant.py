"""What the attention's wrappers make of a decay that is a parameter (no GPU needed)."""
import pytest
import torch

from chunkwise_delta_rule_chunk_amd import ops


def test_a_decay_that_requires_a_gradient():
    """Refused while gradients are recorded, and as good as a constant where they are not."""
    q, g = torch.zeros(1, 8, 4, 64), torch.nn.Parameter(-torch.ones(4))
    with pytest.raises(ValueError, match="no gradient"):
        ops.decay_attention_autograd(q, q, q, g)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ops.decay_attention_autograd(q, q, q, g)
