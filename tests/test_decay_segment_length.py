"""A segment of the attention has at most 32768 tokens, however many sequences and heads fill
the chip: the walks' states carry the decay's rounding once a chunk from its start (no GPU needed)."""
import pytest

from chunkwise_delta_rule_chunk_amd import binding as B


@pytest.mark.parametrize("dtype", [B.REWY_BF16, B.REWY_F32])
@pytest.mark.parametrize("N,T,H", [(1, 1 << 20, 512), (1, 32769, 512), (8, 100000, 64), (1, 40000, 2048)])
def test_segments_of_long_sequences(N, T, H, dtype):
    K = V = 32
    d = B.RewyDecayDesc(N, T, H, 1, K, V, 0, None, None, dtype, 0.1, *[0] * 7)
    segments = N * -(-T // 32768)
    for phase, states in ((0, 1), (1, 2)):
        assert B.rewy_decay_workspace_bytes(d, phase) >= states * segments * H * K * V * 4
    d.T = 32768
    assert B.rewy_decay_workspace_bytes(d, 0) == 256  # one segment each: no states
