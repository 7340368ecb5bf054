"""Heads without channels (no GPU needed)."""
import contextlib

import pytest
import torch

from chunkwise_delta_rule_chunk_amd import binding as B
from chunkwise_delta_rule_chunk_amd import decay_ops, ops


@pytest.mark.parametrize("fn", [ops.decay_attention, ops.decay_attention_recurrent, ops.decay_attention_autograd])
def test_heads_without_channels(fn, monkeypatch):
    """A row length of zero is refused by the entry's own message."""
    monkeypatch.setattr(decay_ops, "_On", lambda *a: contextlib.nullcontext())
    q, v = torch.zeros(1, 8, 4, 0), torch.zeros(1, 8, 4, 64)
    with pytest.raises(B.RewyError):
        fn(q, q, v, -torch.ones(4))
    assert "bad shape K=0" in B.rewy_last_error()
