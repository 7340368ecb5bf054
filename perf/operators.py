"""Cases of the operators around the recurrent token mixer: the RMS norm with
the residual's addition and an 8-bit output, the short causal convolution and
the selective state space scan, each for prompts, for training and for single
tokens.  ``run`` computes them by elementary torch operations, or with ``own``
by the library's kernels."""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ESZ = {"bf16": 2, "fp32": 4}
CHUNK = 64  # tokens per block of the plain scan


# ---- cases -----------------------------------------------------------------
def listed():
    return [
        # one new token for each of 16 sequences: the norm before an 8-bit projection
        dict(name="norm_rows16_d4096_e4m3", op="norm", train=False, M=16, D=4096, dtype="bf16", wdt="bf16",
             residual=True, quant="e4m3", group=0, output=False),
        # a prompt's norm, scales per 128 columns, the 16-bit output kept beside
        dict(name="norm_rows8192_d4096_e4m3_g128", op="norm", train=False, M=8192, D=4096, dtype="bf16",
             wdt="fp32", residual=True, quant="e4m3", group=128, output=True),
        # a training step's norm, forward and backward
        dict(name="norm_train_rows8192_d4096", op="norm", train=True, M=8192, D=4096, dtype="bf16", wdt="fp32",
             residual=True, quant="none", group=0, output=True),
        # rows of an odd length in 32 bits, whole numbers out
        dict(name="norm_rows10007_d1537_fp32_int8", op="norm", train=False, M=10007, D=1537, dtype="fp32",
             wdt="fp32", residual=False, quant="int8", group=0, output=True),
        # a prompt's convolution over x, B and C side by side (32 heads of 128, a state of 128)
        dict(name="conv_t8192_d4352", op="conv", kind="prompt", B=1, T=8192, nseq=0, cut=0, D=4352, W=4, dtype="bf16",
             wdt="bf16", bias=True, silu=True, state=False),
        # a training step over 16 packed sequences of ragged lengths, 16 heads of 128
        dict(name="conv_train_varlen16_d2304", op="conv", kind="train", B=1, T=32768, nseq=16, cut=3, D=2304, W=4,
             dtype="bf16", wdt="fp32", bias=True, silu=True, state=True),
        # one new token for each of 64 sequences
        dict(name="conv_step64_d4352", op="conv", kind="step", B=64, T=1, nseq=0, cut=0, D=4352, W=4, dtype="bf16",
             wdt="bf16", bias=True, silu=True, state=True),
        # a prompt at the width of the delta-rule workload: 32 heads of 128, a state of 128
        dict(name="scan_t8192_h32_n128_p128", op="scan", kind="prompt", B=1, T=8192, nseq=0, cut=0, H=32, G=1, N=128,
             P=128, dtype="bf16", dtd="bf16", state=False),
        # packed ragged sequences in 32 bits, two groups of heads
        dict(name="scan_varlen16_h16_n64_p64_fp32", op="scan", kind="prompt", B=1, T=9000, nseq=16, cut=5, H=16, G=2,
             N=64, P=64, dtype="fp32", dtd="fp32", state=True),
        # a training step on a long sequence
        dict(name="scan_train_t8192_h32_n128_p64", op="scan", kind="train", B=1, T=8192, nseq=0, cut=0, H=32, G=1,
             N=128, P=64, dtype="bf16", dtd="fp32", state=False),
        # a training step in 32 bits, lengths that end inside a block
        dict(name="scan_train_b2_t1000_h16_n64_p64_fp32", op="scan", kind="train", B=2, T=1000, nseq=0, cut=0, H=16,
             G=4, N=64, P=64, dtype="fp32", dtd="fp32", state=True),
        # one new token for each of 64 sequences
        dict(name="scan_step64_h32_n128_p64", op="scan", kind="step", B=64, T=1, nseq=0, cut=0, H=32, G=1, N=128, P=64,
             dtype="bf16", dtd="bf16", state=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    wdt = rng.choice([dtype, "fp32"])
    op = rng.choice(["norm", "conv", "scan", "scan"])
    if op == "norm":
        D = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        M = _log(rng, 1, max(2, 8192 * 4096 // D))
        train = rng.random() < 0.4
        quant = "none" if train else rng.choice(["none", "e4m3", "int8"])
        return dict(op=op, train=train, M=M, D=D, dtype=dtype, wdt=wdt, residual=rng.random() < 0.7, quant=quant,
                    group=rng.choice([0, 128]) if quant != "none" else 0,
                    output=True if train or quant == "none" else rng.random() < 0.5)
    kind = rng.choice(["prompt", "prompt", "train", "train", "step"])
    nseq = rng.choice([0, 0, rng.randint(1, 24)]) if kind != "step" else 0
    if op == "conv":
        D = _log(rng, 32, 4352)
        if rng.random() < 0.6:
            D = max(32, D // 32 * 32)
        B = rng.randint(1, 200) if kind == "step" else 1 if nseq else rng.choice([1, 1, 2, 5])
        T = 1 if kind == "step" else _log(rng, 1, max(4, min(32768, 8192 * 4352 // D) // B))
        return dict(op=op, kind=kind, B=B, T=T, nseq=nseq, cut=rng.randint(0, 999), D=D, W=rng.choice([2, 3, 4, 4]),
                    dtype=dtype, wdt=wdt, bias=rng.random() < 0.7, silu=rng.random() < 0.8,
                    state=kind == "step" or rng.random() < 0.5)
    sizes = [32, 64] if dtype == "fp32" else [32, 64, 128]
    N, P = rng.choice(sizes), rng.choice(sizes)
    G = rng.choice([1, 1, 2, 3, 4])
    H = G * rng.randint(1, max(1, 32 // G))
    B = rng.randint(1, 96) if kind == "step" else 1 if nseq else rng.choice([1, 1, 2, 3])
    most = 8192 * 32 * 128 * 64 // (2 if dtype == "fp32" else 1)
    T = 1 if kind == "step" else _log(rng, 1, max(2, min(16384, most // (H * N * P)) // B))
    return dict(op=op, kind=kind, B=B, T=T, nseq=nseq, cut=rng.randint(0, 999), H=H, G=G, N=N, P=P, dtype=dtype, dtd=wdt,
                state=kind == "step" or rng.random() < 0.5)


def _lens(case):
    """The sequences' lengths: the batch rows, or `nseq` packed ones (some of them may be empty)."""
    if not case["nseq"]:
        return [case["T"]] * case["B"]
    r = random.Random(case["cut"])
    cuts = sorted(r.randint(0, case["T"]) for _ in range(case["nseq"] - 1))
    cuts = [0] + cuts + [case["T"]]
    return [b - a for a, b in zip(cuts, cuts[1:])]


# ---- inputs ----------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def rn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    def ru(*s):
        return torch.rand(*s, generator=gen, device="cuda")

    dt = DT[case["dtype"]]
    st = dict(case)
    if case["op"] == "norm":
        M, D, wdt = case["M"], case["D"], DT[case["wdt"]]
        x = rn(M, D)
        x[:, int(seed) % D] *= 20.0  # one channel of large values
        st.update(x=x.to(dt), r=rn(M, D).mul_(2.0).to(dt) if case["residual"] else None,
                  w=(1.0 + 0.2 * rn(D)).to(wdt))
        if case["train"]:
            st.update(dy=rn(M, D).to(dt), ds=rn(M, D).to(dt) if case["residual"] else None)
        return st
    lens = _lens(case)
    n, B, T = len(lens), case["B"], case["T"]
    cu = None
    if case["nseq"]:
        off = [0]
        for k in lens:
            off.append(off[-1] + k)
        cu = torch.tensor(off, dtype=torch.int32, device="cuda")
    st.update(lens=lens, cu=cu)
    if case["op"] == "conv":
        D, W, wdt = case["D"], case["W"], DT[case["wdt"]]
        st.update(x=rn(B, T, D).to(dt), w=(ru(D, W) - 0.5).mul_(2 * W ** -0.5).to(wdt),
                  b=rn(D).mul_(0.1).to(wdt) if case["bias"] else None,
                  h0=rn(n, W - 1, D).to(dt) if case["state"] else None)
        if case["kind"] == "train":
            st.update(dy=rn(B, T, D).to(dt), dht=rn(n, W - 1, D).to(dt) if case["state"] else None)
        if case["kind"] != "step":
            st.update(plan=_conv_plan(lens, W))
        return st
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    # x, B and C as the convolution leaves them: slices of one row
    row = torch.nn.functional.silu(rn(B, T, H * P + 2 * G * N)).to(dt)
    x, bm, cm = row.split([H * P, G * N, G * N], dim=-1)
    step = torch.exp(ru(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    st.update(x=x.unflatten(-1, (H, P)), bm=bm.unflatten(-1, (G, N)), cm=cm.unflatten(-1, (G, N)),
              dt=rn(B, T, H).to(DT[case["dtd"]]), dt_bias=step + torch.log(-torch.expm1(-step)),
              a_log=torch.log(1.0 + 15.0 * ru(H)), d=1.0 + 0.1 * rn(H),
              h0=rn(n, H, N, P).mul_(0.3) if case["state"] else None)
    if case["kind"] == "train":
        st.update(dy=rn(B, T, H, P).to(dt), dht=rn(n, H, N, P).mul_(0.1) if case["state"] else None)
    if case["kind"] != "step":
        st.update(plan=_scan_plan(lens))
    return st


def _conv_plan(lens, W):
    """Row of [states ; tokens] that each tap of each token reads, and the rows of the final states."""
    idx, fin, t0, ns = [], [], 0, len(lens) * (W - 1)
    for k, n in enumerate(lens):
        # rows of the sequence with its state in front
        rows = torch.cat([torch.arange(k * (W - 1), (k + 1) * (W - 1)), ns + torch.arange(t0, t0 + n)])
        idx.append(rows.unfold(0, W, 1)[:n] if n else rows.new_zeros(0, W))
        fin.append(rows[len(rows) - (W - 1):])
        t0 += n
    return dict(idx=torch.cat(idx).t().contiguous().cuda(), fin=torch.cat(fin).cuda())


def _scan_plan(lens):
    """Tokens of each block (the row behind the last token where it has none), the blocks' sequences, and each
    sequence's first and last block."""
    total, tok, seq, first, last, t0 = sum(lens), [], [], [], [], 0
    for k, n in enumerate(lens):
        first.append(len(seq))
        for a in range(0, n, CHUNK):
            i = torch.arange(a, a + CHUNK)
            tok.append(torch.where(i < n, t0 + i, torch.full_like(i, total)))
            seq.append(k)
        last.append(max(len(seq) - 1, 0))
        t0 += n
    first = [min(i, len(seq) - 1) for i in first]  # an empty sequence has no block of its own
    return dict(tok=torch.stack(tok).cuda(), seq=torch.tensor(seq).cuda(), first=torch.tensor(first).cuda(),
                last=torch.tensor(last).cuda(), some=torch.tensor([n > 0 for n in lens]).cuda())


# ---- one pass --------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def _run_own(st):
    from chunkwise_delta_rule_chunk_amd import ops
    if st["op"] == "norm":
        y, s, q, scale, ctx = ops.rms_norm(st["x"], st["w"], st["r"], eps=1e-6,
                                           quant=None if st["quant"] == "none" else st["quant"],
                                           group=st["group"], output=st["output"])
        out = dict(y=y, s=s if st["residual"] else None, scale=scale, q=_values(q, scale, st["group"]))
        if st["train"]:
            gr = ops.rms_norm_backward(ctx, st["dy"], st["ds"])
            out.update(dx=gr["dx"], dw=gr["dweight"])
        return out
    if st["op"] == "conv":
        act = "silu" if st["silu"] else None
        if st["kind"] == "step":
            y, ht = ops.short_conv_step(st["x"][:, 0], st["h0"], st["w"], st["b"], activation=act)
            return dict(y=y, ht=ht)
        y, ht, ctx = ops.short_conv(st["x"], st["w"], st["b"], activation=act, h0=st["h0"], cu_seqlens=st["cu"],
                                    output_final_state=st["state"])
        out = dict(y=y, ht=ht)
        if st["kind"] == "train":
            gr = ops.short_conv_backward(ctx, st["dy"], st["dht"])
            out.update(dx=gr["dx"], dw=gr["dweight"], db=gr["dbias"], dh0=gr["dh0"])
        return out
    a = (st["x"], st["dt"], st["a_log"], st["bm"], st["cm"])
    kw = dict(d=st["d"], dt_bias=st["dt_bias"], h0=st["h0"])
    if st["kind"] == "step":
        y, ht = ops.selective_scan_recurrent(*a, **kw)
        return dict(y=y, ht=ht)
    y, ht, ctx = ops.selective_scan(*a, **kw, cu_seqlens=st["cu"], output_final_state=st["state"])
    out = dict(y=y, ht=ht)
    if st["kind"] == "train":
        gr = ops.selective_scan_backward(ctx, st["dy"], st["dht"])
        out.update(gr)
    return out


def _run_plain(st):
    if st["op"] == "norm":
        return _norm_plain(st)
    if st["op"] == "conv":
        return _conv_step_plain(st) if st["kind"] == "step" else _conv_plain(st)
    return _scan_step_plain(st) if st["kind"] == "step" else _scan_plain(st)


def _values(q, scale, group):
    """What an 8-bit output stands for, in 16 bits."""
    if q is None:
        return None
    M, D = q.shape
    full = scale if not group else scale.repeat_interleave(group, dim=1)[:, :D]
    return (q.float() * full).to(torch.bfloat16)


def _norm_plain(st):
    dt, D = st["x"].dtype, st["D"]
    s = st["x"].float()
    if st["residual"]:
        s = s + st["r"].float()
    rstd = torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-6)
    w = st["w"].float()
    y = s * rstd * w
    q = scale = None
    if st["quant"] != "none":
        g = st["group"] or D
        ng = -(-D // g)
        yp = torch.nn.functional.pad(y, (0, ng * g - D)).view(-1, ng, g)
        top = 448.0 if st["quant"] == "e4m3" else 127.0
        amax = yp.abs().amax(-1)
        scale = torch.where(amax > 0, amax / top, torch.ones_like(amax))
        v = yp / scale[..., None]
        v = v.to(torch.float8_e4m3fn).float() if st["quant"] == "e4m3" else torch.round(v)
        q = (v * scale[..., None]).view(-1, ng * g)[:, :D].to(torch.bfloat16)
    out = dict(y=y.to(dt) if st["output"] else None, s=s.to(dt) if st["residual"] else None, scale=scale, q=q)
    if st["train"]:
        s = s.to(dt).float()
        dy = st["dy"].float()
        u = dy * w
        dx = rstd * (u - s * (rstd * rstd * (u * s).mean(-1, keepdim=True)))
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        out.update(dx=dx.to(dt), dw=(dy * s * rstd).sum(0).to(st["w"].dtype))
    return out


def _conv_plain(st):
    dt, D, W, plan = st["x"].dtype, st["D"], st["W"], st["plan"]
    x = st["x"].reshape(-1, D).float()
    h0 = st["h0"].reshape(-1, D).float() if st["state"] else x.new_zeros(len(st["lens"]) * (W - 1), D)
    ext, w = torch.cat([h0, x]), st["w"].float()
    idx = list(plan["idx"].unbind(0))
    taps = list(w.unbind(1))
    pre = sum(ext[i] * t for i, t in zip(idx, taps))
    if st["bias"]:
        pre = pre + st["b"].float()
    sig = torch.sigmoid(pre)
    y = pre * sig if st["silu"] else pre
    out = dict(y=y.to(dt).view(st["x"].shape), ht=ext[plan["fin"]].to(dt).view(-1, W - 1, D) if st["state"] else None)
    if st["kind"] == "train":
        dpre = st["dy"].reshape(-1, D).float()
        if st["silu"]:
            dpre = dpre * sig * (1.0 + pre * (1.0 - sig))
        dext = torch.zeros_like(ext)
        if st["state"]:
            dext[plan["fin"]] += st["dht"].reshape(-1, D).float()
        dw = torch.stack([(dpre * ext[i]).sum(0) for i in idx], 1)
        for i, t in zip(idx, taps):
            dext[i] += dpre * t
        ns = h0.shape[0]
        out.update(dx=dext[ns:].to(dt).view(st["x"].shape), dw=dw.to(st["w"].dtype),
                   db=dpre.sum(0).to(st["w"].dtype) if st["bias"] else None,
                   dh0=dext[:ns].to(dt).view(-1, W - 1, D) if st["state"] else None)
    return out


def _conv_step_plain(st):
    dt = st["x"].dtype
    ext = torch.cat([st["h0"].float(), st["x"].float()], 1)  # [n, W, D]
    pre = (ext * st["w"].float().t()).sum(1)
    if st["bias"]:
        pre = pre + st["b"].float()
    y = pre * torch.sigmoid(pre) if st["silu"] else pre
    return dict(y=y.to(dt), ht=ext[:, 1:].to(dt))


def _softplus(z):
    return z.clamp_min(0.0) + torch.log1p(torch.exp(-z.abs()))


def _scan_step_plain(st):
    x, B, H, G = st["x"][:, 0].float(), st["B"], st["H"], st["G"]
    dt = _softplus(st["dt"][:, 0].float() + st["dt_bias"])
    a = torch.exp(-torch.exp(st["a_log"]) * dt)
    bm = st["bm"][:, 0].float().repeat_interleave(H // G, 1)
    cm = st["cm"][:, 0].float().repeat_interleave(H // G, 1)
    S = a[..., None, None] * st["h0"] + (dt[..., None] * bm)[..., None] * x[:, :, None, :]
    y = (S * cm[..., None]).sum(2) + st["d"][:, None] * x
    return dict(y=y.to(st["x"].dtype)[:, None], ht=S)


def _blocks(t, tok):
    """[B, T, H, K] -> [H, blocks, CHUNK, K] in 32 bits, zeros where a block has no token."""
    t = t.float().flatten(0, 1)
    t = torch.cat([t, t.new_zeros(1, *t.shape[1:])])
    return t[tok].permute(2, 0, 1, 3).contiguous()


def _rows(t, tok, shape):
    """[H, blocks, CHUNK, K] -> [B, T, H, K]"""
    out = t.new_empty(shape[0] * shape[1] + 1, t.shape[0], t.shape[3])
    out[tok.reshape(-1)] = t.permute(1, 2, 0, 3).reshape(-1, t.shape[0], t.shape[3])
    return out[:-1].view(*shape[:2], t.shape[0], t.shape[3])


def _scan_plain(st):
    H, G, N, P = st["H"], st["G"], st["N"], st["P"]
    tok, seq, first, last, some = (st["plan"][k] for k in ("tok", "seq", "first", "last", "some"))
    nseq = len(st["lens"])
    nb, odt = tok.shape[0], st["x"].dtype
    h0 = st["h0"] if st["state"] else torch.zeros(nseq, H, N, P, device="cuda")
    X = _blocks(st["x"], tok)
    per = H // G
    Bm = _blocks(st["bm"], tok)
    Cm = _blocks(st["cm"], tok)
    z = st["dt"].float() + st["dt_bias"]
    dt = _blocks(_softplus(z)[..., None], tok)[..., 0]  # [H, nb, 64], zero where there is no token
    A = -torch.exp(st["a_log"])
    g = (A[:, None, None] * dt).double()
    cum = g.cumsum(-1)
    end = cum[..., -1]                                   # [H, nb]
    before = end.cumsum(-1) - end                        # sum over the earlier blocks
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf).float())
    CB = torch.matmul(Cm, Bm.transpose(-1, -2).contiguous()).repeat_interleave(per, 0)
    Bh, Ch = Bm.repeat_interleave(per, 0), Cm.repeat_interleave(per, 0)
    eg, ek = torch.exp(cum.float())[..., None], torch.exp((end[..., None] - cum).float())[..., None]
    dtc = dt[..., None]
    loc = torch.matmul((Bh * (ek * dtc)).transpose(-1, -2).contiguous(), X)  # [H, nb, N, P]
    # the state that enters each block: from the earlier blocks of its sequence and its initial state
    same = seq[:, None] == seq[None, :]
    earlier = same & torch.ones(nb, nb, dtype=torch.bool, device="cuda").tril(-1)
    link = (before[:, :, None] - (before + end)[:, None, :]).masked_fill(~earlier, -math.inf).float().exp()
    into = torch.matmul(link, loc.view(H, nb, -1)).view(H, nb, N, P)
    into += torch.exp((before - before[:, first[seq]]).float())[..., None, None] * h0[seq].transpose(0, 1)
    yin = torch.matmul(Ch, into)
    M = CB * decay * dt[..., None, :]
    Y = torch.matmul(M, X) + eg * yin + st["d"][:, None, None, None] * X
    after = torch.exp(end.float())[..., None, None] * into + loc
    out = dict(y=_rows(Y, tok, st["x"].shape).to(odt), ht=None)
    if st["state"]:
        out["ht"] = torch.where(some[:, None, None, None], after[:, last].transpose(0, 1), h0)
    if st["kind"] != "train":
        return out
    dY = _blocks(st["dy"], tok)
    dht = st["dht"] if st["state"] else torch.zeros_like(h0)
    adj = torch.matmul((Ch * eg).transpose(-1, -2).contiguous(), dY)
    later = torch.matmul(link.transpose(-1, -2).contiguous(), adj.view(H, nb, -1)).view(H, nb, N, P)
    tail = (before + end)[:, last[seq]] - (before + end)
    later += torch.exp(tail.float())[..., None, None] * dht[seq].transpose(0, 1)
    dvin = torch.matmul(Bh, later)
    prod = torch.matmul(dY, X.transpose(-1, -2).contiguous()) * decay
    inner = prod * CB
    rows = ((inner * dt[..., None, :]).sum(-1) + (eg * dY * yin).sum(-1)).double()
    cols = (inner.sum(-2) + (ek * X * dvin).sum(-1)).double()
    diff = rows - dt.double() * cols
    dg = diff.flip(-1).cumsum(-1).flip(-1) + (after.double() * later).sum((-1, -2))[..., None]
    ddt = cols + A.double()[:, None, None] * dg
    dv = torch.matmul((CB * decay).transpose(-1, -2).contiguous(), dY) + ek * dvin
    dX = dtc * dv + st["d"][:, None, None, None] * dY
    Wm = prod * dt[..., None, :]
    dC = torch.matmul(Wm, Bh) + torch.matmul(eg * dY, into.transpose(-1, -2).contiguous())
    dB = torch.matmul(Wm.transpose(-1, -2).contiguous(), Ch) + torch.matmul(ek * dtc * X, later.transpose(-1, -2).contiguous())
    dz = _rows(ddt[..., None], tok, st["x"].shape)[..., 0] * torch.sigmoid(z.double())
    out.update(dx=_rows(dX, tok, st["x"].shape).to(odt), ddt=dz.to(st["dt"].dtype),
               da_log=(dg * g).sum((1, 2)).float(),
               db=_rows(dB.view(G, per, nb, CHUNK, N).sum(1), tok, st["x"].shape).to(odt),
               dc=_rows(dC.view(G, per, nb, CHUNK, N).sum(1), tok, st["x"].shape).to(odt),
               dd=(X.double() * dY).sum((1, 2, 3)).float(), ddt_bias=dz.sum((0, 1)).float(), dh0=None)
    if st["state"]:
        dh0 = (torch.exp(end.float())[..., None, None] * later + adj)[:, first].transpose(0, 1)
        out["dh0"] = torch.where(some[:, None, None, None], dh0, dht)
    return out


# ---- what one pass cannot do without -----------------------------------------
def work(case):
    e = ESZ[case["dtype"]]
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        rows = 1 + (2 if case["residual"] else 0) + (1 if case["output"] else 0)  # x, r and s, y
        b, f = M * D * e * rows + D * ESZ[case["wdt"]], 4 * M * D
        if case["quant"] != "none":
            b += M * D + 4 * M * (-(-D // case["group"]) if case["group"] else 1)
            f += 3 * M * D
        if case["train"]:
            b += M * D * e * (3 if case["residual"] else 2) + D * ESZ[case["wdt"]]  # dy, ds, dx
            f += 9 * M * D
        return dict(bytes=b, flops=f)
    n, tok = case["nseq"] or case["B"], case["B"] * case["T"]
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        par = D * (W + (1 if case["bias"] else 0)) * ESZ[case["wdt"]]
        st = 2 * n * (W - 1) * D * e if case["state"] else 0
        b, f = 2 * tok * D * e + par + st, tok * D * (2 * W + 4)
        if case["kind"] == "train":
            b, f = b + 2 * tok * D * e + par + st, f + tok * D * (4 * W + 8)
        return dict(bytes=b, flops=f)
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    st = 2 * n * H * N * P * 4 if case["state"] else 0
    b = tok * (2 * H * P * e + 2 * G * N * e + H * ESZ[case["dtd"]]) + 12 * H + st
    f = 4 * tok * H * N * P
    if case["kind"] == "train":
        b += tok * (2 * H * P * e + 2 * G * N * e + H * ESZ[case["dtd"]]) + 12 * H + st
        f += 10 * tok * H * N * P
    return dict(bytes=b, flops=f)


# ---- the definitions in 64 bits ----------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(st)
    if case["op"] == "conv":
        return _conv_exact(st)
    return _scan_exact(st)


def _norm_exact(st):
    leaf = st["x"].double() + (st["r"].double() if st["residual"] else 0.0)
    w = st["w"].double()
    norm = (leaf.square().sum(-1, keepdim=True) / st["D"] + 1e-6).sqrt()
    y = leaf / norm * w
    q = scale = None
    if st["quant"] != "none":
        top, g = (448.0, 127.0)[st["quant"] == "int8"], st["group"] or st["D"]
        qs, ss = [], []
        for a in range(0, st["D"], g):
            part = y[:, a:a + g]
            k = part.abs().max(1, keepdim=True).values / top
            k = torch.where(k > 0, k, torch.ones_like(k))
            if st["quant"] == "int8":
                v = (part / k).round()
            else:  # nearest multiple of 2^(e-3), e the exponent, at least -6
                m = part / k
                ex = torch.frexp(m.abs().clamp_min(2.0 ** -6)).exponent.double() - 4
                v = (m / torch.exp2(ex)).round() * torch.exp2(ex)
            qs.append(v * k)
            ss.append(k)
        q, scale = torch.cat(qs, 1), torch.cat(ss, 1)
    out = dict(y=y if st["output"] else None, s=leaf if st["residual"] else None, scale=scale, q=q)
    if st["train"]:
        # the backward's row is the sum as it is kept, its statistic the forward's
        row = leaf.to(st["x"].dtype).double() if st["residual"] else leaf
        u = st["dy"].double() * w
        dx = u / norm - row / norm ** 3 * (u * row).sum(-1, keepdim=True) / st["D"]
        if st["ds"] is not None:
            dx = dx + st["ds"].double()
        out.update(dx=dx, dw=torch.einsum("md,md->d", st["dy"].double(), row / norm))
    return out


def _conv_exact(st):
    D, W = st["D"], st["W"]
    x = st["x"].double().flatten(0, 1).requires_grad_(st["kind"] == "train")
    w = st["w"].double().requires_grad_(st["kind"] == "train")
    b = st["b"].double().requires_grad_(st["kind"] == "train") if st["bias"] else None
    n = len(st["lens"])
    h0 = (st["h0"].double() if st["state"] else torch.zeros(n, W - 1, D, device="cuda").double())
    h0 = h0.requires_grad_(st["kind"] == "train")
    ys, hts, t0 = [], [], 0
    for k, ln in enumerate(st["lens"]):
        seq = torch.cat([h0[k], x[t0:t0 + ln]])
        pre = torch.zeros(ln, D, device="cuda").double()
        for j in range(W):
            pre = pre + seq[j:j + ln] * w[:, j]
        if b is not None:
            pre = pre + b
        ys.append(pre / (1.0 + torch.exp(-pre)) if st["silu"] else pre)
        hts.append(seq[ln:])
        t0 += ln
    y, ht = torch.cat(ys), torch.stack(hts)
    out = dict(y=y.detach().view(st["x"].shape), ht=ht.detach() if st["state"] else None)
    if st["kind"] == "step":
        out["y"] = out["y"][:, 0]
    if st["kind"] == "train":
        loss = (y * st["dy"].double().flatten(0, 1)).sum()
        if st["state"]:
            loss = loss + (ht * st["dht"].double()).sum()
        wrt = [x, w, h0] + ([b] if b is not None else [])
        gr = torch.autograd.grad(loss, wrt, allow_unused=True)
        out.update(dx=gr[0].view(st["x"].shape), dw=gr[1], db=gr[3] if b is not None else None,
                   dh0=gr[2] if st["state"] else None)
    return out


def _scan_exact(st):
    """Token by token; sequences side by side, the shorter ones keeping their state."""
    H, G, N, P = st["H"], st["G"], st["N"], st["P"]
    lens, n = st["lens"], len(st["lens"])
    most, per = max(lens), H // G
    train = st["kind"] == "train"
    if most > 20000 or (train and most * n * H * N * P * 8 > 48 << 30):
        return None
    tot = sum(lens)
    tok = torch.full((most, n), tot, dtype=torch.long)
    t0 = 0
    for k, ln in enumerate(lens):
        tok[:ln, k] = torch.arange(t0, t0 + ln)
        t0 += ln
    tok = tok.cuda()

    def by_time(t):
        t = t.double().flatten(0, 1)
        return torch.cat([t, t.new_zeros(1, *t.shape[1:])])[tok]  # [most, n, ...]

    x = by_time(st["x"])
    bm, cm = (by_time(st[k]).repeat_interleave(per, 2) for k in ("bm", "cm"))
    live = (tok < tot).double()[..., None]
    z = by_time(st["dt"]) + st["dt_bias"].double()
    dt = torch.nn.functional.softplus(z, threshold=60.0) * live
    a = torch.exp(-torch.exp(st["a_log"].double()) * dt)
    d = st["d"].double()
    S = st["h0"].double() if st["state"] else torch.zeros(n, H, N, P, device="cuda").double()
    keep = torch.empty(most + 1, n, H, N, P, device="cuda", dtype=torch.float64) if train else None
    y = torch.empty_like(x)
    for t in range(most):
        if train:
            keep[t] = S
        S = a[t][..., None, None] * S + (dt[t][..., None] * bm[t])[..., None] * x[t][:, :, None, :]
        y[t] = torch.matmul(cm[t][:, :, None, :], S)[:, :, 0]
    y = y + d[:, None] * x

    def by_token(t, like):
        out = t.new_zeros(tot + 1, *t.shape[2:])
        out[tok.reshape(-1)] = t.flatten(0, 1)
        return out[:-1].reshape(like.shape)

    res = dict(y=by_token(y, st["x"]), ht=S if st["state"] else None)
    if not train:
        return res
    keep[most] = S
    dy = by_time(st["dy"])
    dS = st["dht"].double() if st["state"] else torch.zeros_like(S)
    dx, db, dc = torch.empty_like(x), torch.empty_like(bm), torch.empty_like(cm)
    ddt, dlog = torch.empty_like(dt), torch.empty_like(dt)
    for t in range(most - 1, -1, -1):
        dc[t] = torch.matmul(keep[t + 1], dy[t][..., None])[..., 0]
        dS = dS + cm[t][..., None] * dy[t][:, :, None, :]
        dv = torch.matmul(bm[t][:, :, None, :], dS)[:, :, 0]
        db[t] = torch.matmul(dS, (dt[t][..., None] * x[t])[..., None])[..., 0]
        dx[t] = dt[t][..., None] * dv
        ddt[t] = (dv * x[t]).sum(-1)
        dS = a[t][..., None, None] * dS
        dlog[t] = (dS * keep[t]).sum((-1, -2))
    A = -torch.exp(st["a_log"].double())
    dz = (ddt + A * dlog) * torch.sigmoid(z) * live
    dx = dx + d[:, None] * dy
    grp = lambda t: t.view(most, n, G, per, N).sum(3)  # noqa: E731
    res.update(dx=by_token(dx, st["x"]), ddt=by_token(dz, st["dt"]), da_log=(dlog * A * dt).sum((0, 1)),
               db=by_token(grp(db), st["bm"]), dc=by_token(grp(dc), st["cm"]), dd=(x * dy).sum((0, 1, 3)),
               ddt_bias=dz.sum((0, 1)), dh0=dS if st["state"] else None)
    return res
