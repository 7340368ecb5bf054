"""Sizes at which the operators around the token mixer run their main loops more than once:
several heads a workgroup in the scan's chunk backward (even and uneven ranges), segments
of 512 tokens and decay chains over their eight chunks, segments joined at K = V = 128,
runs of 32 and 64 tokens in the convolution, more rows than blocks in the norm's backward.
Each case says which of the host's choices it is for and checks, from the sizes of the
workspaces, that the host still makes them.

Bounds of the scan: as derived in test_ssm_gpu.py; the sums over the heads add at most 32
additions to the 64 + 128 that its 300 U hold.
Convolution: a term of dweight or dbias is within 30 U of its magnitude; then ``run``
additions in a register, ceil(tiles / 16) in a group and 16 joins.
Norm: a lane sums n = 16 .. 32 squares, then 6 joins in the wave and at most 16 waves one after
another: (n + 22) U for the sum, half of it for the root and 3 U for mean, root and division, so
30 U for rstd; y and the terms below take 4 roundings more.  dweight: ceil(M / rows at once) rows
in a register, at most 16 joins in the block, 16 + 64 over the blocks."""
import pytest
import torch

from layer_util import DT, U32, close
from parity_util import gpu_available, say
from test_conv_gpu import _formula as conv_formula, _inputs as conv_inputs
from test_norm_gpu import EPS, _formula as norm_formula, _inputs as norm_inputs
from test_ssm_gpu import _check_backward, _check_forward, _cu, _inputs, _references

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU and librewy.so")]


def _up(n):
    return -(-n // 256) * 256


def _scan_bytes(B, T, H, G, K, V, n, fp32, packed, bwd, seg, split):
    """Bytes of the scan's workspace with segments of ``seg`` tokens and ``split`` head ranges."""
    total = B * T
    slots = lambda L: total // L + n if packed else n * max(-(-T // L), 1)  # noqa: E731
    nslot, nchunk, kv, e, tok = slots(seg), slots(64), H * K * V, 4 if fp32 else 2, H * total * 4
    parts = [nchunk * H * 64 * 16, nchunk * G * 10 * 256 * 4]
    if (total if packed else T) > seg:
        parts += [nslot * kv * 4] * (2 if bwd else 1) + [2 * nslot * H * 4]
    if bwd:
        parts += [nchunk * kv * e] * 2 + [tok, tok, 2 * tok, 2 * tok, nchunk * H * 16, tok, nslot * H * 8, nchunk * H * 4,
                                          nchunk * H * 4, nchunk * 2 * H * 8]
        if split > 1:
            parts.append(2 * split * total * G * K * 4)
    return sum(_up(p) for p in parts)


def _scan_choice(desc, n, bwd):
    """(tokens of a segment, head ranges) that give the workspace its size."""
    from chunkwise_delta_rule_chunk_amd import binding as B
    need = B.rewy_ssm_workspace_bytes(desc, int(bwd))
    packed, fp32 = bool(desc.cu_seqlens), desc.dtype == B.REWY_F32
    longest = desc.B * desc.T if packed else desc.T
    found = set()
    most = 512 if bwd and not fp32 else max(longest, 256)  # (the bf16 backward's longest)
    for seg in range(256, most + 64, 64):
        for split in range(1, 33 if bwd else 2):
            if _scan_bytes(desc.B, desc.T, desc.H, desc.G, desc.K, desc.V, n, fp32, packed, bwd, seg, split) == need:
                found.add((min(seg, longest), split))
    return found


SCANS = [
    # B, T, H, G, K, V, dtype, lens, state, decay, segment (backward), head ranges (backward)
    (4, 1000, 128, 4, 32, 32, "bf16", None, True, "usual", 512, 1),     # 32 heads each, segments of 512
    (4, 1000, 128, 4, 32, 32, "bf16", None, True, "none", 512, 1),      # ... no chunk that decays: chains of 8 chunks
    (1, 1100, 32, 1, 128, 128, "bf16", None, True, "usual", 256, 11),   # 2 or 3 heads each
    (1, 1100, 32, 1, 128, 64, "bf16", None, False, "usual", 256, 11),
    (1, 1100, 32, 1, 64, 64, "bf16", None, True, "usual", 256, 11),     # 16 waves
    (1, 1100, 32, 1, 64, 128, "bf16", None, True, "strong", 256, 11),
    (1, 1100, 32, 1, 64, 64, "fp32", None, True, "usual", 256, 11),
    (1, 1200, 40, 2, 32, 64, "fp32", [500, 0, 613, 1, 86], True, "usual", 256, 5),
    (1, 1200, 48, 2, 128, 32, "bf16", [1, 700, 63, 64, 372], True, "usual", 256, 5),   # 4 or 5 heads each
    (1, 1300, 4, 1, 128, 128, "bf16", [600, 700], True, "none", 256, 4),
]


@pytest.mark.parametrize("case", SCANS, ids=["_".join(str(v) for v in c[:7]) + ("_packed" if c[7] else "") + "_" + c[9] for c in SCANS])
def test_scan(case):
    from chunkwise_delta_rule_chunk_amd import ops
    B, T, H, G, K, V, dtype, lens, state, decay, seg, split = case
    say(f"[case] {case}")
    ln = lens or [T] * B
    args, kw, dy, dht = _inputs(B, T, H, G, K, V, dtype, "fp32", T + K + V, len(ln), state, decay)
    y, ht, ctx = ops.selective_scan(*args, **kw, cu_seqlens=_cu(lens, T))
    assert _scan_choice(ctx["desc"], len(ln), True) == {(seg, split)}
    ref, mag = _references(args, kw, ln, dy, dht)
    _check_forward(y, ht, ref, mag, max(ln), dtype)
    gr = ops.selective_scan_backward(ctx, dy, dht)
    torch.cuda.synchronize()
    _check_backward(gr, ref, mag, args, kw, ln, dy, dht, dtype)


def _conv_choice(desc):
    """(tokens of a run of the backward, runs); the forward's runs have half as many, at most 32."""
    from chunkwise_delta_rule_chunk_amd import binding as B
    need, total = B.rewy_conv_workspace_bytes(desc), desc.B * desc.T
    found = {run: -(-total // run) for run in (4, 8, 16, 32, 64) if _up(-(-total // run) * (desc.W + 1) * desc.D * 4) == need}
    assert len(found) == 1
    return next(iter(found.items()))


ENDS = [0, 1, 2, 3, 0, 4, 63, 64, 65, 31, 32, 33, 7, 5000, 0]


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,dtype,wdt,packed", [(1028, "bf16", "fp32", True), (1030, "bf16", "bf16", True),
                                                (1028, "fp32", "fp32", False), (1027, "fp32", "bf16", True)])
def test_convolution(W, D, dtype, wdt, packed):
    """Runs of 64 tokens (the forward's of 32), with channels in whole and in partial vectors."""
    from chunkwise_delta_rule_chunk_amd import ops
    T = 32800
    lens = ENDS + [T - sum(ENDS)] if packed else [T]
    x, w, b, h0, dy, dht = conv_inputs(1, T, D, W, dtype, wdt, D + W, len(lens))
    y, ht, ctx = ops.short_conv(x, w, b, h0=h0, cu_seqlens=_cu(lens if packed else None, T), output_final_state=True)
    run, tiles = _conv_choice(ctx["desc"])
    assert run == 64 and T % run  # the last run is a partial one
    gr = ops.short_conv_backward(ctx, dy, dht)
    ref = conv_formula(x, w, b, h0, dy, dht, True, lens)
    close(y[0], ref["y"], 16 * U32 * (ref["mag"] + ref["y"].abs()), "y")
    close(ht, ref["ht"], 0.0, "ht")
    # dx_t = sum over the taps of dpre, each within 20 U of its magnitude, by the same sum
    aw, reach = w.double().abs(), torch.zeros_like(ref["dx"])
    hreach, t0 = torch.zeros(len(lens), W - 1, D, dtype=torch.float64, device="cuda"), 0
    for k, n in enumerate(lens):
        ext = torch.zeros(n + W - 1, D, dtype=torch.float64, device="cuda")
        for j in range(W):  # token i reaches row i + j of [state ; tokens] by tap j
            ext[j:j + n] += ref["dmag"][t0:t0 + n] * aw[:, j]
        hreach[k], reach[t0:t0 + n] = ext[:W - 1], ext[W - 1:]
        t0 += n
    dh = dht.double().abs().max()
    close(gr["dx"][0], ref["dx"], 30 * U32 * (reach + dh), "dx")
    close(gr["dh0"], ref["dh0"], 30 * U32 * (hreach + dh), "dh0")
    steps = 30 + run + -(-tiles // 16) + 16
    close(gr["dweight"], ref["dweight"], steps * U32 * (ref["dmag"] * ref["tap"]).sum(1).t(), "dweight")
    close(gr["dbias"], ref["dbias"], steps * U32 * ref["dmag"].sum(0), "dbias")


@pytest.mark.parametrize("M,D,dtype,rows", [(2600, 2048, "bf16", 1), (3100, 5000, "bf16", 1), (2300, 16384, "bf16", 1),
                                            (2300, 16383, "fp32", 1), (2500, 3001, "fp32", 1), (9000, 500, "bf16", 4),
                                            (40000, 120, "bf16", 16)])
def test_norm_backward(M, D, dtype, rows):
    """Every block takes several rows (``rows`` at once)."""
    from chunkwise_delta_rule_chunk_amd import binding as B
    from chunkwise_delta_rule_chunk_amd import ops
    x, r, w = norm_inputs(M, D, dtype, "fp32", M + D)
    desc = B.RewyNormDesc(M, D, B.REWY_F32 if dtype == "fp32" else B.REWY_BF16, B.REWY_F32, 0, 0, EPS, 0, 0, 0, 0)
    blocks = 1024
    assert B.rewy_norm_workspace_bytes(desc) == _up(blocks * D * 4) and M > 2 * blocks * rows
    y, s, _, _, ctx = ops.rms_norm(x, w, r, eps=EPS)
    s64, rstd, y64 = norm_formula(x, r, w)
    close(y, y64, 40 * U32 * y64.abs(), "y")
    close(s, s64, U32 * s64.abs(), "s")
    close(ctx["rstd"], rstd[:, 0], 30 * U32 * rstd[:, 0], "rstd")
    g = torch.Generator().manual_seed(7)
    dy, ds = (torch.randn(M, D, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    gr = ops.rms_norm_backward(ctx, dy, ds)
    row, k = s.double(), ctx["rstd"].double()[:, None]  # the backward's own inputs
    u = dy.double() * w.double()
    dx = k * (u - row * (u * row).mean(-1, keepdim=True) * k * k) + ds.double()
    # the row's dot sums terms of both signs: 32 in a lane, 6 + 16 joins, and 6 products around it
    mag = k * (u.abs() + row.abs() * (u * row).abs().mean(-1, keepdim=True) * k * k) + ds.double().abs()
    close(gr["dx"], dx, 60 * U32 * mag, "dx")
    terms = dy.double() * row * k
    steps = -(-M // (blocks * rows)) + 16 + 16 + 64 + 3
    close(gr["dweight"], terms.sum(0), steps * U32 * terms.abs().sum(0), "dweight")
