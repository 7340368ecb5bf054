"""Outputs of the attention with a constant decay that share bytes with an input or another
output are refused, wherever they begin; slices of one row that lie between each other are
not (no GPU needed: what passes is stopped by a workspace that is too small, or not called)."""
import ctypes
import random

import pytest

from chunkwise_delta_rule_chunk_amd import binding as B

P = ctypes.c_void_p
BASE = 1 << 40
H, G, K, V, T = 4, 2, 64, 32, 10
ROW = {"q": H * K * 2, "k": G * K * 2, "v": G * V * 2, "o": H * V * 2, "dO": H * V * 2, "dq": H * K * 2, "dk": G * K * 2,
       "dv": G * V * 2}  # bytes


def _at(v):
    return None if v is None else P(v)


def _far():
    """Addresses of every tensor, none near another."""
    names = ("q", "k", "v", "o", "dO", "dq", "dk", "dv", "h0", "ht", "dht", "dh0", "g", "ws", "states")
    return {n: BASE + (i << 30) for i, n in enumerate(names)}


def _desc(strides, tokens=T, seqs=1):
    s = [strides.get(n, 0) // 2 for n in ("q", "k", "v", "o", "dq", "dk", "dv")]
    return B.RewyDecayDesc(seqs, tokens, H, G, K, V, 0, None, None, B.REWY_BF16, 0.1, *s)


def fwd(at, strides=None, **kw):
    d = _desc(strides or {}, **kw)
    return B.rewy_decay_fwd(d, *(_at(at[n]) for n in ("q", "k", "v", "g", "h0", "o", "ht", "ws")), 1 << 40, None)


def step(at, strides=None, **kw):
    d = _desc(strides or {}, **kw)
    return B.rewy_decay_recurrent_fwd(d, *(_at(at[n]) for n in ("q", "k", "v", "g", "h0", "o", "ht")), None)


def bwd(at, strides=None, **kw):
    d = _desc(strides or {}, **kw)
    return B.rewy_decay_bwd(d, *(_at(at[n]) for n in ("q", "k", "v", "g", "h0", "dO", "dht")), None, 0,
                            *(_at(at[n]) for n in ("dq", "dk", "dv", "dh0", "ws")), 1 << 40, None)


STATE = H * K * V * 4


@pytest.mark.parametrize("call,name,other,off", [
    (fwd, "o", "q", ROW["q"] * T - 16), (fwd, "o", "k", -(ROW["o"] * T) + 16), (fwd, "o", "v", 16),
    (fwd, "ht", "h0", 16), (fwd, "ht", "h0", -STATE + 16), (fwd, "o", "h0", STATE - 16), (fwd, "ht", "o", 64),
    (fwd, "ht", "g", -STATE + 16),
    (step, "o", "q", 32), (step, "ht", "h0", 16), (step, "ht", "h0", 16 - STATE), (step, "ht", "v", 0),
    (bwd, "dq", "q", 16), (bwd, "dk", "dq", ROW["dq"] * T - 16), (bwd, "dv", "dk", -16), (bwd, "dv", "dO", 16),
    (bwd, "dh0", "dht", 16), (bwd, "dh0", "h0", -16), (bwd, "dq", "dh0", 16), (bwd, "dv", "h0", 0), (bwd, "dk", "v", 16),
])
def test_a_shared_byte_is_refused(call, name, other, off):
    at = _far()
    at[name] = at[other] + off
    assert call(at) == B.REWY_EINVAL and "overlaps" in B.rewy_last_error()
    assert name in B.rewy_last_error() and other in B.rewy_last_error()


def _slices(order, row, shift=None):
    """Places of the named tensors one behind the other in rows of `row` bytes."""
    at, x = _far(), BASE + (100 << 30)
    for n in order:
        at[n] = x
        x += ROW[n]
    if shift:
        at[shift[0]] += shift[1]
    return at, {n: row for n in order}


@pytest.mark.parametrize("shift", [("dk", -16), ("dq", 16), ("dv", 16), ("dk", -2048 + 16), ("dv", 2048 * 3 + 16), None])
def test_slices_of_one_row(shift):
    """The gradients' joint row: exact slices are apart, a slice that is 16 bytes too early or
    too late is not, in whatever row."""
    at, st = _slices(("dq", "dk", "dv"), ROW["dq"] + ROW["dk"] + ROW["dv"], shift)
    at["dh0"] = at["dht"] + 16  # (refused for this at the latest)
    assert bwd(at, st) == B.REWY_EINVAL
    assert ("dh0 overlaps dht" in B.rewy_last_error()) == (shift is None)


# What passes goes on to the GPU, so the rule itself is looked at beside a plain one that
# marks every byte, through a call whose other pointers are bad.
def test_the_rule_against_marked_bytes():
    """Random rows at random strides: refused exactly when a byte is shared.  A state that
    overlaps its own adjoint stops the calls that are right."""
    rng = random.Random(3)
    seen = [0, 0]
    for _ in range(3000):
        tokens = rng.choice([1, 2, 3, 7])
        wide = lambda n: rng.choice([0, ROW[n], ROW[n] + 16 * rng.randint(0, 40), 2 * ROW[n] + 16 * rng.randint(0, 8)])  # noqa: E731
        st = {n: wide(n) for n in ("dq", "dv")}
        if rng.random() < 0.3:
            st["dq"] = st["dv"] = ROW["dq"] + ROW["dv"] + 16 * rng.randint(0, 4)
        at = _far()
        at["dv"] = at["dq"] + 16 * rng.randint(-120, 120)
        at["dh0"] = at["dht"] + 16

        def marked(n):
            s = st[n] or ROW[n]
            return {(at[n] + t * s + i) // 16 for t in range(tokens) for i in range(0, ROW[n], 16)}

        shared = bool(marked("dq") & marked("dv"))
        assert bwd(at, st, tokens=tokens) == B.REWY_EINVAL
        if at["dq"] == at["dv"]:
            continue  # (refused by its own rule)
        got = B.rewy_last_error()
        assert ("dv overlaps dq" in got) == shared, (st, tokens, at["dv"] - at["dq"], got)
        assert shared or "dh0 overlaps dht" in got
        seen[shared] += 1
    assert min(seen) > 200
