"""The selective state space mixer's operators, as they are measured: the scan
(`ssm_fwd`, `ssm_bwd`, `ssm_step`), its short convolution with bias, SiLU and a
carried state (`conv_silu`, `conv_silu_bwd`, `conv_silu_step`) and the gated
norm behind a mixer (`gated_norm`, `gated_norm_bwd`).

`own` chooses between the framework's kernels and a plain form of elementary
torch operations in 32 bits; `exact` computes the same from the definitions in
64 bits, token by token.  A case is a dict of plain values; `op` is one of

    scan_train  forward and backward of the scan        (bf16)
    scan        forward of the scan, a prompt           (bf16)
    scan_step   one token of every sequence             (bf16 or fp32)
    conv_train  forward and backward of the convolution
    conv        forward of the convolution, a prompt
    conv_step   one token of every sequence
    norm_train  forward and backward of the gated norm
    norm        forward of the gated norm

`seqs` > 0 packs that many sequences of uneven lengths into the T tokens (B is
1 then); `state` gives a carried state (h0 or the convolution's last inputs).
"""
import math
import random

import torch

own = False

CHUNK = 64  # tokens per chunk of the plain scan


def _case(op, dtype="bf16", B=1, T=1, H=1, G=1, dk=0, dv=0, seqs=0, state=False, **more):
    return dict(op=op, dtype=dtype, B=B, T=T, H=H, G=G, dk=dk, dv=dv, seqs=seqs, state=state, **more)


def listed():
    cases = {
        # a training step's micro-batch of a state space layer: all heads share one key and one query
        "scan train 4x4096": _case("scan_train", B=4, T=4096, H=32, G=1, dk=128, dv=64),
        # a short ragged pack with odd lengths, grouped keys, carried states
        "scan train ragged": _case("scan_train", T=1357, H=6, G=2, dk=64, dv=128, seqs=9, state=True),
        # one long prompt: few streams, so the sequence itself has to be split
        "scan prompt 1x16384": _case("scan", T=16384, H=16, G=16, dk=128, dv=128),
        # a server's packed prefill with states carried from earlier pieces
        "scan packed 65536": _case("scan", T=65536, H=32, G=8, dk=128, dv=128, seqs=8, state=True),
        # decoding at a full batch: the state's traffic
        "scan step 256": _case("scan_step", B=256, H=32, G=8, dk=128, dv=128, state=True),
        # decoding for one user: latency
        "scan step 1": _case("scan_step", "fp32", B=1, H=8, G=1, dk=64, dv=64, state=True),
        # the convolution in front of the scan, training
        "conv train 4x4096": _case("conv_train", B=4, T=4096, H=32, dv=128, W=4),
        # a ragged pack continued from carried inputs, odd channel count, fp32
        "conv packed ragged": _case("conv", "fp32", T=3001, H=5, dv=40, seqs=7, state=True, W=3),
        # the convolution of a decoding batch
        "conv step 256": _case("conv_step", B=256, H=32, dv=128, state=True, W=4),
        # the norm behind the recurrence, per head, training
        "norm train 4x4096": _case("norm_train", B=4, T=4096, H=16, dv=256, first=False, shared=True),
        # the norm over a whole wide row with the gate inside it, fp32
        "norm train wide": _case("norm_train", "fp32", B=2, T=1001, H=2, dv=2048, first=True, shared=False),
        # the norm of a decoding batch
        "norm decode 256": _case("norm", B=256, T=1, H=32, dv=128, first=False, shared=True),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["scan_train", "scan", "scan_step", "conv_train", "conv", "conv_step", "norm_train", "norm"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("scan"):
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
        G = rng.choice([g for g in range(1, H + 1) if H % g == 0])
        dk, dv = rng.choice([64, 128]), 64 * rng.choice([1, 1, 2, 2, 3, 4])
        if op == "scan_step":
            return _case(op, kind, B=_log(rng, 1, max(1, 256 * 32 * 128 // (H * dv))), H=H, G=G, dk=dk, dv=dv, state=True)
        top = (16384 * 32 * 64 if op == "scan_train" else 65536 * 32 * 128) // (H * dv + G * dk)
        T = _log(rng, 1, min(top, 65536))
        if rng.random() < 0.4:
            return _case(op, T=T, H=H, G=G, dk=dk, dv=dv, seqs=rng.randint(1, 12), state=rng.random() < 0.5)
        return _case(op, B=max(1, min(_log(rng, 1, 16), top // T)), T=T, H=H, G=G, dk=dk, dv=dv, state=rng.random() < 0.5)
    H, dv = _log(rng, 1, 32), 8 * _log(rng, 1, 32)
    if op.startswith("conv"):
        W = rng.choice([2, 3, 4])
        if op == "conv_step":
            return _case(op, kind, B=_log(rng, 1, 256), H=H, dv=dv, state=True, W=W)
        T = _log(rng, 1, 16384 * 32 * 128 // (H * dv) if H * dv > 4096 else 16384)
        if rng.random() < 0.4:
            return _case(op, kind, T=T, H=H, dv=dv, seqs=rng.randint(1, 12), state=rng.random() < 0.5, W=W)
        return _case(op, kind, B=max(1, min(_log(rng, 1, 8), 16384 // T)), T=T, H=H, dv=dv, state=rng.random() < 0.5, W=W)
    T = _log(rng, 1, 16384 * 16 * 256 // (H * dv) if H * dv > 4096 else 16384)
    return _case(op, kind, T=T, H=H, dv=dv * rng.choice([1, 1, 1, 16]) if T < 1024 else dv, first=rng.random() < 0.5,
                 shared=rng.random() < 0.5)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _lengths(case):
    """The sequences' lengths: B times T, or a pack's uneven ones (its shape alone decides them)."""
    if not case["seqs"]:
        return [case["T"]] * case["B"]
    rng = random.Random(case["T"] * 131 + case["seqs"])
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def _starts(lens):
    return torch.tensor([0] + lens).cumsum(0)


def prepare(case, seed):
    dev, E, op = _device(), _dtype(case), case["op"]
    gen = torch.Generator(dev).manual_seed(int(seed))
    n01 = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    B, T, H, G, dk, dv = (case[k] for k in ("B", "T", "H", "G", "dk", "dv"))
    lens = _lengths(case)
    N = len(lens)
    s = dict(case=case, cu=None)
    if op.endswith("_step"):
        N, lead = B, (B,)
    else:
        lead = (B, T)
        cu = _starts(lens)
        s["lens"] = lens
        s["cu"] = cu.to(torch.int32).to(dev) if case["seqs"] else None
        # each token's sequence, and its place in it
        s["seq"] = torch.repeat_interleave(torch.arange(N), torch.tensor(lens)).to(dev)
        s["pos"] = torch.arange(B * T, device=dev) - cu.to(dev)[s["seq"]]
        s["len"] = torch.tensor(lens).to(dev)
    silu = lambda x: x * torch.sigmoid(x)  # noqa: E731
    if op.startswith("scan"):
        # what the short convolution and SiLU leave; step sizes as a state space layer sets them up
        s["q"], s["k"] = silu(n01(*lead, G, dk)).to(E), silu(n01(*lead, G, dk)).to(E)
        s["v"] = silu(n01(*lead, H, dv)).to(E)
        s["dt"] = n01(*lead, H)
        step = torch.exp(uni(H) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -(1 + 15 * uni(H))
        s["skip"] = 1 + 0.1 * n01(H)
        s["h0"] = 0.1 * n01(N, H, dk, dv) if case["state"] else None
        if op == "scan_train":
            s["dO"] = n01(B, T, H, dv).to(E)
            s["dhT"] = 0.1 * n01(N, H, dk, dv) if case["state"] else None
        if not op.endswith("_step"):
            # the plain form's plan: chunks of 64 tokens that restart at every sequence; row BT stands for padding
            rows, of = [], []
            for n, (at, ln) in enumerate(zip(_starts(lens).tolist(), lens)):
                for c in range(0, ln, CHUNK):
                    m = min(CHUNK, ln - c)
                    rows.append([at + c, m])
                    of.append(n)
            r = torch.tensor(rows, dtype=torch.int64).reshape(-1, 2).to(dev)
            i = torch.arange(CHUNK, device=dev)
            s["rows"] = torch.where(i < r[:, 1:], r[:, :1] + i, B * T)
            s["of"] = torch.tensor(of, dtype=torch.int64).to(dev)
            s["back"] = torch.empty(B * T + 1, dtype=torch.int64, device=dev)
            s["back"][s["rows"].reshape(-1)] = torch.arange(s["rows"].numel(), device=dev)
            s["back"] = s["back"][: B * T]
    elif op.startswith("conv"):
        W = case["W"]
        s["x"] = n01(*lead, H, dv).to(E)
        s["w"] = n01(H, dv, W) / math.sqrt(W)
        s["bias"] = 0.1 * n01(H, dv)
        s["s0"] = n01(N, W - 1, H, dv).to(E) if case["state"] else None
        if op == "conv_train":
            s["dy"] = n01(*lead, H, dv).to(E)
            s["dsT"] = n01(N, W - 1, H, dv).to(E) if case["state"] else None
    else:
        s["x"], s["z"] = n01(B, T, H, dv).to(E), n01(B, T, H, dv).to(E)
        s["w"] = 1 + 0.1 * (n01(dv) if case["shared"] else n01(H, dv))
        if op == "norm_train":
            s["dy"] = n01(B, T, H, dv).to(E)
    return s


EPS = 1e-5


def _run_own(s):
    import chunkwise_delta_rule_wy_amd as dn
    c = s["case"]
    op = c["op"]
    if op == "scan_step":
        o = dn.ssm_step(s["q"], s["k"], s["v"], s["dt"], s["A"], s["bias"], s["skip"], s["h0"])
        return dict(o=o, state=s["h0"])
    if op.startswith("scan"):
        o, hT = dn.ssm_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["bias"], s["skip"], s["h0"], s["cu"])
        if op == "scan":
            return dict(o=o, hT=hT)
        g = dn.ssm_bwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["bias"], s["skip"], s["h0"], s["dO"], s["dhT"], s["cu"])
        if s["h0"] is None:
            g.pop("dh0")
        return dict(g, o=o, hT=hT)
    if op == "conv_step":
        y = dn.conv_silu_step(s["x"], s["w"], s["bias"], s["s0"])
        return dict(y=y, state=s["s0"])
    if op.startswith("conv"):
        y, sT = dn.conv_silu(s["x"], s["w"], s["bias"], s["s0"], s["cu"])
        if op == "conv":
            return dict(y=y, sT=sT)
        g = dn.conv_silu_bwd(s["x"], s["w"], s["bias"], s["s0"], s["dy"], s["dsT"], s["cu"])
        if s["s0"] is None:
            g.pop("ds0")
        return dict(g, y=y, sT=sT)
    y = dn.gated_norm(s["x"], s["z"], s["w"], eps=EPS, gate_first=c["first"])
    if op == "norm":
        return dict(y=y)
    dx, dz, dw = dn.gated_norm_bwd(s["x"], s["z"], s["w"], s["dy"], eps=EPS, gate_first=c["first"])
    return dict(y=y, dx=dx, dz=dz, dw=dw)


def _softplus(x):
    return torch.relu(x) + torch.log1p(torch.exp(-x.abs()))


def _scan_plain(s, q, k, v, dt, A, bias, skip, h0):
    """The chunk form of the scan over the plan's chunks, in 32 bits (log decays in 64): inside a chunk every
    pair of tokens, between chunks every pair of chunks of one sequence."""
    c = s["case"]
    H, G, dk, dv = c["H"], c["G"], c["dk"], c["dv"]
    rows, of, N = s["rows"], s["of"], len(s["lens"])
    NC = rows.shape[0]

    def chunks(x):  # [B, T, heads, d] -> [chunk, heads, 64, d], padding rows zero
        x = x.reshape(-1, x.shape[-2], x.shape[-1])
        return torch.cat([x, x.new_zeros(1, *x.shape[1:])])[rows].transpose(1, 2).contiguous()

    step = _softplus(dt + bias)
    sc = chunks(step[..., None])[..., 0]                                # [NC, H, 64]
    b = (sc.double() * A.double()[:, None]).cumsum(-1)
    i = torch.arange(CHUNK, device=b.device)
    decay = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(i[:, None] < i, -torch.inf)).float()
    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    p = (qc @ kc.transpose(-1, -2)).repeat_interleave(H // G, 1) * decay * sc[..., None, :]
    kh, qh = kc.repeat_interleave(H // G, 1), qc.repeat_interleave(H // G, 1)
    add = kh.transpose(-1, -2) @ (vc * (torch.exp(b[..., -1:] - b).float() * sc)[..., None])
    # decay from the end of chunk j to the start of chunk i, both of one sequence
    total = b[..., -1].transpose(0, 1)                                  # [H, NC]
    upto = total.cumsum(-1)
    same = (of[:, None] == of) & (torch.arange(NC, device=of.device)[:, None] > torch.arange(NC, device=of.device))
    link = torch.exp((upto[:, :, None] - total[:, :, None] - upto[:, None, :]).masked_fill(~same, -torch.inf)).float()
    start = (link @ add.transpose(0, 1).reshape(H, NC, dk * dv)).reshape(H, NC, dk, dv).transpose(0, 1)
    # the last chunk of each sequence, from which its final state follows
    has = s["len"] > 0
    ends = (torch.arange(N, device=of.device)[:, None] == of).cumsum(1).argmax(1) if NC else s["len"]
    if h0 is not None:
        first = (torch.arange(N, device=of.device)[:, None] == of).long().argmax(1) if NC else s["len"]
        since = upto - total - (upto - total)[:, first[of]] if NC else upto
        start = start + torch.exp(since).float().transpose(0, 1)[..., None, None] * h0[of]
    y = p @ vc + torch.exp(b).float()[..., None] * (qh @ start)
    o = y.transpose(1, 2).reshape(-1, H, dv)[s["back"]].reshape(v.shape) + skip[:, None] * v
    end = torch.exp(b[..., -1]).float()[..., None, None] * start + add
    empty = h0 if h0 is not None else v.new_zeros(N, H, dk, dv)
    hT = torch.where(has[:, None, None, None], end[ends], empty) if NC else empty
    return o, hT


def _step_plain(s):
    c, E = s["case"], _dtype(s["case"])
    R = c["H"] // c["G"]
    q, k = (s[n].float().repeat_interleave(R, 1) for n in ("q", "k"))
    v, step = s["v"].float(), _softplus(s["dt"] + s["bias"])
    h = torch.exp(step * s["A"])[..., None, None] * s["h0"] + k[..., :, None] * (step[..., None] * v)[..., None, :]
    o = (q[..., None] * h).sum(-2) + s["skip"][:, None] * v
    s["h0"].copy_(h)
    return dict(o=o.to(E), state=s["h0"])


def _conv_taps(s, x, s0):
    """Each token's W inputs [tokens, W, channels]: earlier tokens of its sequence, before them the carried ones (or zeros)."""
    W, C = s["case"]["W"], x.shape[-1]
    j = torch.arange(W, device=x.device)
    at = s["pos"][:, None] - (W - 1) + j                               # place in the sequence
    n = x.shape[0]
    row = torch.where(at >= 0, torch.arange(n, device=x.device)[:, None] - (W - 1) + j, n + s["seq"][:, None] * (W - 1) + at + W - 1)
    return torch.cat([x, s0.reshape(-1, C)])[row]


def _conv_plain(s):
    c, E = s["case"], _dtype(s["case"])
    W, H, dv, N = c["W"], c["H"], c["dv"], len(s["lens"])
    C = H * dv
    x = s["x"].float().reshape(-1, C)
    s0 = s["s0"].float().reshape(N, W - 1, C) if s["s0"] is not None else x.new_zeros(N, W - 1, C)
    w, bias = s["w"].reshape(C, W), s["bias"].reshape(C)
    taps = _conv_taps(s, x, s0)
    z = (taps * w.t()).sum(1) + bias
    sig = torch.sigmoid(z)
    shape = s["x"].shape
    # the final state: the last W - 1 inputs of [carried, tokens] of each sequence
    start = _starts(s["lens"])[:-1].to(x.device)
    at = s["len"][:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
    n = x.shape[0]
    last = torch.where(at >= 0, start[:, None] + at, n + torch.arange(N, device=x.device)[:, None] * (W - 1) + at + W - 1)
    out = dict(y=(z * sig).to(E).reshape(shape), sT=torch.cat([x, s0.reshape(-1, C)])[last].to(E).reshape(N, W - 1, H, dv))
    if c["op"] == "conv":
        return out
    dz = s["dy"].float().reshape(-1, C) * sig * (1 + z * (1 - sig))
    out["dw"] = (taps * dz[:, None]).sum(0).t().reshape(H, dv, W)
    out["dbias"] = dz.sum(0).reshape(H, dv)
    # an input at place p (carried ones at -(W - 1) .. -1) feeds the outputs p .. p + W - 1 of its sequence
    j = torch.arange(W, device=x.device)
    dzp = torch.cat([dz, dz.new_zeros(1, C)])

    def fed(place, first, length):  # [inputs], rows of dz that each tap's input feeds
        to = place[:, None] + (W - 1) - j
        return torch.where((to >= 0) & (to < length[:, None]), first[:, None] + to, n)

    dx = (dzp[fed(s["pos"], start[s["seq"]], s["len"][s["seq"]])] * w.t()).sum(1)
    places = torch.arange(-(W - 1), 0, device=x.device).repeat(N)
    own_seq = torch.arange(N, device=x.device).repeat_interleave(W - 1)
    ds0 = (dzp[fed(places, start[own_seq], s["len"][own_seq])] * w.t()).sum(1)
    both = torch.cat([dx, ds0])
    if s["dsT"] is not None:
        both = both.index_add(0, last.reshape(-1), s["dsT"].float().reshape(-1, C))
    out["dx"] = both[:n].to(E).reshape(shape)
    if s["s0"] is not None:
        out["ds0"] = both[n:].to(E).reshape(N, W - 1, H, dv)
    return out


def _conv_step_plain(s):
    E = _dtype(s["case"])
    line = torch.cat([s["s0"], s["x"][:, None]], 1).float()            # [B, W, H, D]
    z = (line * s["w"].permute(2, 0, 1)).sum(1) + s["bias"]
    s["s0"].copy_(line[:, 1:])
    return dict(y=(z * torch.sigmoid(z)).to(E), state=s["s0"])


def _norm_plain(s):
    c, E = s["case"], _dtype(s["case"])
    x, z, w = s["x"].float(), s["z"].float(), s["w"]
    sig = torch.sigmoid(z)
    gate = z * sig
    u = x * gate if c["first"] else x
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    n = u * r
    y = n * w if c["first"] else n * w * gate
    if c["op"] == "norm":
        return dict(y=y.to(E))
    dy = s["dy"].float()
    dn = dy * w if c["first"] else dy * w * gate
    du = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dsilu = sig * (1 + z * (1 - sig))
    dx, dz = (du * gate, du * x * dsilu) if c["first"] else (du, dy * w * n * dsilu)
    dw = dy * n if c["first"] else dy * n * gate
    dw = dw.sum((0, 1, 2)) if c["shared"] else dw.sum((0, 1))
    return dict(y=y.to(E), dx=dx.to(E), dz=dz.to(E), dw=dw)


SCAN_GRADS = ("q", "k", "v", "dt", "A", "bias", "skip", "h0")
NAMES = {"q": "dq", "k": "dk", "v": "dv", "dt": "ddt", "A": "dA", "bias": "ddt_bias", "skip": "dskip", "h0": "dh0"}


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["case"]["op"]
    if op == "scan_step":
        return _step_plain(s)
    if op == "conv_step":
        return _conv_step_plain(s)
    if op.startswith("conv"):
        return _conv_plain(s)
    if op.startswith("norm"):
        return _norm_plain(s)
    E = _dtype(s["case"])
    args = {n: (s[n].float() if s[n] is not None else None) for n in SCAN_GRADS}
    if op == "scan":
        o, hT = _scan_plain(s, **args)
        return dict(o=o.to(E), hT=hT)
    given = [n for n in SCAN_GRADS if args[n] is not None]
    args = {n: (args[n].detach().requires_grad_() if args[n] is not None else None) for n in SCAN_GRADS}
    with torch.enable_grad():
        o, hT = _scan_plain(s, **args)
    grads = torch.autograd.grad([o, hT], [args[n] for n in given],
                                [s["dO"].float(), s["dhT"] if s["dhT"] is not None else torch.zeros_like(hT)])
    out = {NAMES[n]: g.to(E) if n in "qkv" else g for n, g in zip(given, grads)}
    return dict(out, o=o.detach().to(E), hT=hT.detach())


def work(case):
    B, T, H, G, dk, dv, op = (case[k] for k in ("B", "T", "H", "G", "dk", "dv", "op"))
    e = 2 if case["dtype"] == "bf16" else 4
    N = case["seqs"] or B
    n = B * T
    if op.startswith("scan"):
        st = 4 * N * H * dk * dv
        rows = n * (2 * G * dk + 2 * H * dv) * e + 4 * n * H
        keep = st * (2 if case["state"] else 1)
        if op != "scan_train":  # a state's update and its product with the query
            return dict(bytes=rows + keep, flops=4.0 * n * H * dk * dv)
        # q, k, v, dt, dO in; o and the gradients out; the adjoint's state, its products with q, k and v
        rows = n * (4 * G * dk + 4 * H * dv) * e + 8 * n * H
        return dict(bytes=rows + keep * (2 if case["state"] else 1), flops=12.0 * n * H * dk * dv)
    C = H * dv
    if op.startswith("conv"):
        W = case["W"]
        st = N * (W - 1) * C * e * (2 if case["state"] else 1)
        if op == "conv_train":
            return dict(bytes=4 * n * C * e + 2 * st + 8 * C * (W + 1), flops=6.0 * n * C * W)
        return dict(bytes=2 * n * C * e + st + 4 * C * (W + 1), flops=2.0 * n * C * W)
    wb = 4 * (dv if case["shared"] else C)
    if op == "norm_train":
        return dict(bytes=6 * n * C * e + 2 * wb, flops=30.0 * n * C)
    return dict(bytes=3 * n * C * e + wb, flops=10.0 * n * C)


def _exact_scan(s):
    """Token by token in 64 bits, all sequences side by side, and the adjoint of that loop."""
    c = s["case"]
    H, G, dk, dv = c["H"], c["G"], c["dk"], c["dv"]
    lens, N, R = s["lens"], len(s["lens"]), c["H"] // c["G"]
    L, dev = max(lens), s["v"].device
    back = s["seq"] * L + s["pos"]

    def lay(x):  # [B, T, ...] -> [L, N, ...], zeros behind the shorter sequences
        y = torch.zeros(N * L, *x.shape[2:], dtype=torch.float64, device=dev)
        y[back] = x.reshape(-1, *x.shape[2:]).double()
        return y.reshape(N, L, *x.shape[2:]).transpose(0, 1).contiguous()

    def unlay(y, like):
        return y.transpose(0, 1).reshape(N * L, *y.shape[2:])[back].reshape(*like.shape[:2], *y.shape[2:])

    raw = s["dt"].double() + s["bias"].double()
    one = lay(torch.logaddexp(raw, torch.zeros_like(raw)))               # step sizes, zero in padding
    A = s["A"].double()
    q, k, v = lay(s["q"]), lay(s["k"]), lay(s["v"])
    h = s["h0"].double() if s["h0"] is not None else torch.zeros(N, H, dk, dv, dtype=torch.float64, device=dev)
    train = c["op"] == "scan_train"
    kept, o = [], torch.zeros(L, N, H, dv, dtype=torch.float64, device=dev)
    for t in range(L):
        if train:
            kept.append(h)
        kt, qt = (x[t].repeat_interleave(R, 1) for x in (k, q))
        h = torch.exp(one[t] * A)[..., None, None] * h + kt[..., None] * (one[t][..., None] * v[t])[:, :, None]
        o[t] = torch.matmul(qt[:, :, None], h)[:, :, 0]
    skip = s["skip"].double()
    out = dict(o=unlay(o, s["v"]) + skip[:, None] * s["v"].double(), hT=h)
    if not train:
        return out
    dO = lay(s["dO"])
    dh = s["dhT"].double() if s["dhT"] is not None else torch.zeros_like(h)
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    done, dlog = torch.zeros_like(one), torch.zeros_like(one)
    for t in reversed(range(L)):
        kt, qt = (x[t].repeat_interleave(R, 1) for x in (k, q))
        dq[t] = torch.matmul(h, dO[t][..., None])[..., 0].reshape(N, G, R, dk).sum(2)
        dh = dh + qt[..., None] * dO[t][:, :, None]
        u = torch.matmul(dh, v[t][..., None])[..., 0]
        dk_[t] = (one[t][..., None] * u).reshape(N, G, R, dk).sum(2)
        done[t] = (kt * u).sum(-1)
        dv_[t] = one[t][..., None] * torch.matmul(kt[:, :, None], dh)[:, :, 0]
        dh = torch.exp(one[t] * A)[..., None, None] * dh
        h = kept.pop()
        dlog[t] = (dh * h).sum((-1, -2))
    dstep = unlay(done + A * dlog, s["dt"])
    ddt = dstep * torch.sigmoid(raw)
    d64 = s["dO"].double()
    out.update(dq=unlay(dq, s["q"]), dk=unlay(dk_, s["k"]), dv=unlay(dv_, s["v"]) + skip[:, None] * d64, ddt=ddt,
               dA=(one * dlog).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dskip=(d64 * s["v"].double()).sum((0, 1, 3)))
    if s["h0"] is not None:
        out["dh0"] = dh
    return out


def _exact_conv(s):
    """One sequence after another in 64 bits, tap by tap; gradients by differentiating that."""
    c = s["case"]
    W, train = c["W"], c["op"] == "conv_train"
    f64 = {n: s[n].double().requires_grad_(train) if s[n] is not None else None for n in ("x", "w", "bias", "s0")}
    x = f64["x"].reshape(-1, c["H"], c["dv"])
    ys, lasts, at = [], [], 0
    with torch.set_grad_enabled(train):
        for n, ln in enumerate(s["lens"]):
            line = torch.cat([f64["s0"][n] if f64["s0"] is not None else x.new_zeros(W - 1, c["H"], c["dv"]), x[at:at + ln]])
            z = f64["bias"] + sum(f64["w"][:, :, j] * line[j:j + ln] for j in range(W))
            ys.append(z / (1 + torch.exp(-z)))
            lasts.append(line[ln:])
            at += ln
        y, sT = torch.cat(ys).reshape(s["x"].shape), torch.stack(lasts)
    out = dict(y=y.detach(), sT=sT.detach())
    if train:
        given = [n for n in ("x", "w", "bias", "s0") if f64[n] is not None]
        up = s["dsT"].double() if s["dsT"] is not None else torch.zeros_like(sT)
        grads = torch.autograd.grad([y, sT], [f64[n] for n in given], [s["dy"].double(), up])
        out.update({"d" + n: g for n, g in zip(given, grads)})
    return out


def _exact_norm(s):
    c = s["case"]
    train = c["op"] == "norm_train"
    x, z, w = (s[n].double().requires_grad_(train) for n in ("x", "z", "w"))
    with torch.set_grad_enabled(train):
        gate = z / (1 + torch.exp(-z))
        u = x * gate if c["first"] else x
        y = u / torch.sqrt(u.pow(2).sum(-1, keepdim=True) / c["dv"] + EPS) * w
        y = y if c["first"] else y * gate
    out = dict(y=y.detach())
    if train:
        out.update(zip(("dx", "dz", "dw"), torch.autograd.grad(y, [x, z, w], s["dy"].double())))
    return out


def exact(case, seed):
    if case["op"] == "scan_train" and max(_lengths(case)) * len(_lengths(case)) * case["H"] * case["dk"] * case["dv"] > 6e9:
        return None  # the loop keeps every state
    if case["op"] in ("scan", "scan_train") and max(_lengths(case)) > (40000 if case["op"] == "scan" else 20000):
        return None  # too long a loop
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan_step":
        h0 = s["h0"]
        R = case["H"] // case["G"]
        raw = s["dt"].double() + s["bias"].double()
        one = torch.logaddexp(raw, torch.zeros_like(raw))
        k, q = (s[n].double().repeat_interleave(R, 1) for n in ("k", "q"))
        v = s["v"].double()
        h = torch.exp(one * s["A"].double())[..., None, None] * h0.double() + torch.matmul(k[..., None], (one[..., None] * v)[:, :, None])
        o = torch.matmul(q[:, :, None], h)[:, :, 0]
        return dict(o=o + s["skip"].double()[:, None] * v, state=h)
    if op == "conv_step":
        W = case["W"]
        line = torch.cat([s["s0"].double(), s["x"].double()[:, None]], 1)
        z = s["bias"].double() + sum(s["w"].double()[:, :, j] * line[:, j] for j in range(W))
        return dict(y=z / (1 + torch.exp(-z)), state=line[:, 1:])
    return _exact_scan(s) if op.startswith("scan") else _exact_conv(s) if op.startswith("conv") else _exact_norm(s)
