"""The operators around the token mixers, as they are measured: the gated linear
recurrence (`glr_fwd`, `glr_bwd`, `glr_step`), the residual's addition with
dropout and root-mean-square norm (`add_norm`, `add_norm_bwd`), the same norm with
its rows in 8 bits (`norm8`) and the product of such rows with 8-bit weights
(`linear8`).

`own` chooses between the framework's kernels and a plain form of elementary
torch operations in 32 bits; `exact` computes the same from the definitions in
64 bits, written apart.  A case is a dict of plain values; `op` is one of

    glr_train   forward and backward of the recurrence  (B sequences of T tokens,
    glr         forward, a prompt                        H heads of D channels)
    glr_step    one token of every sequence
    norm_train  forward and backward of the addition, dropout and norm (T rows of D)
    norm8       rows in 8 bits
    linear8     M rows times N columns over K

`seqs` > 0 packs that many sequences of uneven lengths into the T tokens (B is
1 then); `state` gives a carried state.
"""
import math
import random

import torch

own = False

POWER = 8.0
EPS = 1e-5
TOP8 = 448.0  # the largest value of an 8-bit float with 4 exponent and 3 mantissa bits


def _glr(op, dtype="bf16", B=1, T=1, H=1, D=8, seqs=0, state=False):
    return dict(op=op, dtype=dtype, B=B, T=T, H=H, D=D, seqs=seqs, state=state)


def _norm(op, T, D, dtype="bf16", wide=False, p=0.0):
    return dict(op=op, dtype=dtype, T=T, D=D, wide=wide, p=p)


def _linear(M, N, K, act="none", bias=False, residual=False):
    return dict(op="linear8", M=M, N=N, K=K, act=act, bias=bias, residual=residual)


def listed():
    cases = {
        # a training step's micro-batch of a recurrent layer
        "recurrence train 4x4096": _glr("glr_train", B=4, T=4096, H=16, D=256),
        # a short ragged pack with odd lengths and channels, carried states, fp32
        "recurrence train ragged": _glr("glr_train", "fp32", T=1357, H=5, D=104, seqs=9, state=True),
        # one long prompt: the sequence itself has to be split
        "recurrence prompt 1x16384": _glr("glr", T=16384, H=16, D=128),
        # a decoding batch: latency
        "recurrence step 256": _glr("glr_step", B=256, H=32, D=128, state=True),
        # the residual stream in front of a layer, training with dropout
        "add norm train 16384": _norm("norm_train", 16384, 4096, p=0.1),
        # a ragged number of odd rows, the residual kept in fp32
        "add norm train ragged": _norm("norm_train", 1357, 520, wide=True),
        # a server's prefill: rows for the 8-bit projections
        "norm8 prompt 16384": _norm("norm8", 16384, 4096),
        # the rows of a decoding batch: latency
        "norm8 decode 256": _norm("norm8", 256, 4096),
        # the projections in front of a mixer, prefill: keys, queries, values and gates
        "linear8 prompt 16384": _linear(16384, 8192, 4096),
        # a ragged prefill into an odd number of columns
        "linear8 ragged 1357": _linear(1357, 1001, 2064, act="gelu", bias=True),
        # the output projection of a decoding batch, added to the residual stream
        "linear8 decode 64": _linear(64, 4096, 4096, residual=True),
        # one user's token: the weights' traffic
        "linear8 decode 1": _linear(1, 8192, 4096, act="silu", bias=True),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["glr_train", "glr", "glr_step", "norm_train", "norm8", "linear8", "linear8"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op == "linear8":
        # serving: a token to a long prefill, columns of one narrow to several wide projections
        N, K = _log(rng, 1, 16384), 16 * _log(rng, 1, 512)
        M = _log(rng, 1, min(16384, 16384 * 8192 * 4096 // (N * K)))
        return _linear(M, N, K, rng.choice(["none", "silu", "gelu"]), rng.random() < 0.5, rng.random() < 0.5)
    if op.startswith("glr"):
        H, D = _log(rng, 1, 32), 8 * _log(rng, 1, 32)
        if op == "glr_step":
            return _glr(op, kind, B=_log(rng, 1, 256), H=H, D=D, state=True)
        top = 4 * 4096 * 16 * 256 // (H * D) // (2 if kind == "fp32" else 1)
        T = _log(rng, 1, min(top, 32768))
        if rng.random() < 0.4:
            return _glr(op, kind, T=T, H=H, D=D, seqs=rng.randint(1, 12), state=rng.random() < 0.5)
        return _glr(op, kind, B=max(1, min(_log(rng, 1, 16), top // T)), T=T, H=H, D=D, state=rng.random() < 0.5)
    D = 8 * _log(rng, 4, 1024)
    T = _log(rng, 1, 16384 * 4096 // D // (2 if kind == "fp32" else 1))
    return _norm(op, T, D, kind, wide=rng.random() < 0.5, p=rng.choice([0.0, 0.1, 0.25]) if op == "norm_train" else 0.0)


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
    dev, op = _device(), case["op"]
    gen = torch.Generator(dev).manual_seed(int(seed))
    n01 = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    s = dict(case=case)
    if op == "linear8":
        M, N, K = case["M"], case["N"], case["K"]

        def rows(x):  # 8-bit rows with a scale each, as a norm's output or a weight matrix is kept
            scale = x.abs().amax(1) / TOP8
            return (x / scale[:, None]).to(torch.float8_e4m3fn), scale

        s["x"], s["xs"] = rows(n01(M, K))
        s["w"], s["ws"] = rows(n01(N, K) / math.sqrt(K))
        s["bias"] = 0.1 * n01(N) if case["bias"] else None
        s["residual"] = n01(M, N).to(torch.bfloat16) if case["residual"] else None
        return s
    E = _dtype(case)
    if op.startswith("glr"):
        B, T, H, D = (case[k] for k in "BTHD")
        lens = _lengths(case)
        N, lead = (B, (B,)) if op == "glr_step" else (len(lens), (B, T))
        # what a short convolution leaves, and two gates' projections
        s["x"], s["r"], s["i"] = n01(*lead, H, D).to(E), n01(*lead, H, D).to(E), n01(*lead, H, D).to(E)
        # decays of 0.9 to 0.999 a token where the gate is open, as such a layer is set up
        keep = 0.9 + 0.099 * torch.rand(H, D, generator=gen, device=dev)
        s["lam"] = torch.log(torch.expm1(-torch.log(keep) / POWER))
        s["br"], s["bi"] = 0.1 * n01(H, D), 0.1 * n01(H, D)
        s["h0"] = n01(N, H, D) if case["state"] else None
        if op == "glr_train":
            s["dy"] = n01(B, T, H, D).to(E)
            s["dhT"] = n01(N, H, D) if case["state"] else None
        if op != "glr_step":
            cu = _starts(lens)
            s["lens"] = lens
            s["cu"] = cu.to(torch.int32).to(dev) if case["seqs"] else None
            # each token's sequence, its place in it, and the tokens behind it
            s["seq"] = torch.repeat_interleave(torch.arange(N), torch.tensor(lens)).to(dev)
            s["pos"] = torch.arange(B * T, device=dev) - cu.to(dev)[s["seq"]]
            s["len"] = torch.tensor(lens).to(dev)
            s["left"] = s["len"][s["seq"]] - 1 - s["pos"]
        return s
    T, D, R = case["T"], case["D"], torch.float32 if case["wide"] else E
    s["x"], s["res"] = n01(T, D).to(E), n01(T, D).to(R)
    s["w"] = 1 + 0.1 * n01(D)
    # the dropout's key and the number of its stream (a layer's, a step's)
    s["seed"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=gen, device=dev) if case["p"] else None
    if op == "norm_train":
        s["dy"], s["dh"] = n01(T, D).to(E), n01(T, D).to(R)
    return s


def _run_own(s):
    import chunkwise_delta_rule_wy_amd as dn
    c = s["case"]
    op = c["op"]
    if op == "linear8":
        return dict(y=dn.linear8(s["x"], s["xs"], s["w"], s["ws"], s["bias"], s["residual"], act=c["act"]))
    if op == "glr_step":
        y = dn.glr_step(s["x"], s["r"], s["i"], s["lam"], s["br"], s["bi"], s["h0"], power=POWER)
        return dict(y=y, state=s["h0"])
    if op.startswith("glr"):
        states = dn.glr_states(s["x"]) if op == "glr_train" else None
        y, hT = dn.glr_fwd(s["x"], s["r"], s["i"], s["lam"], s["br"], s["bi"], s["h0"], s["cu"], power=POWER, states=states)
        if op == "glr":
            return dict(y=y, hT=hT)
        g = dn.glr_bwd(s["x"], s["r"], s["i"], s["lam"], s["br"], s["bi"], s["h0"], s["dy"], s["dhT"], s["cu"], power=POWER,
                       states=states)
        if s["h0"] is None:
            g.pop("dh0")
        return dict(g, y=y, hT=hT)
    if op == "norm8":
        y, scale, h = dn.norm8(s["x"], s["res"], s["w"], eps=EPS)
        return dict(y=y, scale=scale, h=h)
    y, h = dn.add_norm(s["x"], s["res"], s["w"], eps=EPS, p=c["p"], seed=s["seed"])
    dx, dres, dw = dn.add_norm_bwd(h, s["w"], s["dy"], s["dh"], eps=EPS, p=c["p"], seed=s["seed"])
    return dict(y=y, h=h, dx=dx, dres=dres, dw=dw)


def _softplus(x):
    return torch.relu(x) + torch.log1p(torch.exp(-x.abs()))


def _gates(s, x, r, i):
    """(log decay, decay, input's factor m, input gate, input) of rows of H D channels, in 32 bits."""
    sr, si = torch.sigmoid(r + s["br"].reshape(-1)), torch.sigmoid(i + s["bi"].reshape(-1))
    log = -POWER * _softplus(s["lam"].reshape(-1)) * sr
    m = torch.sqrt(-torch.expm1(2 * log))
    return log, torch.exp(log), m, sr, si, m * si * x


def _linear_scan(a, b, reach, longest, back):
    """h_t = a_t h_{t -+ 1} + b_t over the `reach[t]` < `longest` tokens before (or behind) t, by doubling; and the product of a over them."""
    step, n = 1, a.shape[0]
    while step < longest:
        at = torch.arange(n, device=a.device) + (step if back else -step)
        has = (reach >= step)[:, None]
        at = at.clamp(0, n - 1)
        b = torch.where(has, a * b[at] + b, b)
        a = torch.where(has, a * a[at], a)
        step *= 2
    return b, a


def _glr_plain(s):
    c, E = s["case"], _dtype(s["case"])
    H, D = c["H"], c["D"]
    C, N = H * D, len(s["lens"])
    x, r, i = (s[k].float().reshape(-1, C) for k in ("x", "r", "i"))
    log, a, m, sr, si, u = _gates(s, x, r, i)
    h0 = s["h0"].reshape(N, C) if s["h0"] is not None else x.new_zeros(N, C)
    h, since = _linear_scan(a, u, s["pos"], max(s["lens"]), False)
    h = h + since * h0[s["seq"]]
    end = _starts(s["lens"])[1:].to(x.device) - 1
    some = (s["len"] > 0)[:, None]
    out = dict(y=h.to(E).reshape(s["x"].shape), hT=torch.where(some, h[end], h0).reshape(N, H, D))
    if c["op"] == "glr":
        return out
    dhT = s["dhT"].reshape(N, C) if s["dhT"] is not None else x.new_zeros(N, C)
    dy = s["dy"].float().reshape(-1, C)
    last = (s["left"] == 0)[:, None]
    after = torch.where(last, 0, torch.cat([a[1:], a[:1]]))  # the next token's decay
    g, _ = _linear_scan(after, dy + torch.where(last, dhT[s["seq"]], 0), s["left"], max(s["lens"]), True)
    before = torch.where((s["pos"] == 0)[:, None], h0[s["seq"]], torch.cat([h[:1], h[:-1]]))
    # dlog of m = sqrt(1 - a^2) is -a^2 / m; the log decay times it stays finite
    dlog = log * (g * a * before) - g * si * x * a * a * torch.where(m > 0, log / m, 0)
    dr = (1 - sr) * dlog
    di = g * m * x * si * (1 - si)
    start = _starts(s["lens"])[:-1].to(x.device).clamp(max=x.shape[0] - 1)
    lam = s["lam"].reshape(-1)
    out.update(dx=(g * m * si).to(E).reshape(s["x"].shape), dr=dr.to(E).reshape(s["x"].shape), di=di.to(E).reshape(s["x"].shape),
               dlam=(dlog.sum(0) * torch.sigmoid(lam) / _softplus(lam)).reshape(H, D), dbr=dr.sum(0).reshape(H, D),
               dbi=di.sum(0).reshape(H, D))
    if s["h0"] is not None:
        out["dh0"] = torch.where(some, (a * g)[start], dhT).reshape(N, H, D)
    return out


def _glr_step_plain(s):
    E = _dtype(s["case"])
    n, C = s["x"].shape[0], s["lam"].numel()
    x, r, i = (s[k].float().reshape(n, C) for k in ("x", "r", "i"))
    _, a, _, _, _, u = _gates(s, x, r, i)
    h = a * s["h0"].reshape(n, C) + u
    s["h0"].copy_(h.reshape(s["h0"].shape))
    return dict(y=h.to(E).reshape(s["x"].shape), state=s["h0"])


MASK32 = 0xFFFFFFFF


def _keep(s, T, D):
    """The dropout's factors [T, D]: 0 or 1 / (1 - p).  Random bits by Philox4x32 with 7 rounds (Salmon et al., "Parallel
    random numbers: as easy as 1, 2, 3", 2011): one block of 4 words for 8 values, 16 bits each."""
    drop = round(s["case"]["p"] * 65536)
    key, stream = s["seed"][0], s["seed"][1]
    unit = torch.arange(T * D // 8, device=s["seed"].device)
    c = [unit & MASK32, unit >> 32, (stream & MASK32).expand_as(unit), ((stream >> 32) & MASK32).expand_as(unit)]
    k0, k1 = key & MASK32, (key >> 32) & MASK32
    for _ in range(7):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]  # 64-bit products; the sign bit is one of their bits
        c = [((p1 >> 32) & MASK32) ^ c[1] ^ k0, p1 & MASK32, ((p0 >> 32) & MASK32) ^ c[3] ^ k1, p0 & MASK32]
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    words = torch.stack(c, 1)
    half = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(T, D)
    return torch.where(half >= drop, 65536.0 / (65536 - drop), 0.0)


def _norm_plain(s):
    c, E = s["case"], _dtype(s["case"])
    x, w = s["x"].float(), s["w"]
    keep = _keep(s, c["T"], c["D"]) if c["p"] else None
    # the sum is rounded as it is stored, and the norm taken of that
    h = (s["res"].float() + (x * keep if keep is not None else x)).to(s["res"].dtype)
    f = h.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    n = f * r
    y = n * w
    if c["op"] == "norm8":
        scale = y.abs().amax(-1).clamp(min=1e-30) / TOP8
        return dict(y=(y / scale[:, None]).to(torch.float8_e4m3fn), scale=scale, h=h)
    dy = s["dy"].float()
    dn = dy * w
    dres = s["dh"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dx = dres * keep if keep is not None else dres
    return dict(y=y.to(E), h=h, dx=dx.to(E), dres=dres.to(h.dtype), dw=(dy * n).sum(0))


def _linear_plain(s):
    z = torch.mm(s["x"].float(), s["w"].float().t()) * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        z = z + s["bias"]
    if s["case"]["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif s["case"]["act"] == "gelu":
        z = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return dict(y=z.to(torch.bfloat16))


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "linear8":
        return _linear_plain(state)
    if op == "glr_step":
        return _glr_step_plain(state)
    return _glr_plain(state) if op.startswith("glr") else _norm_plain(state)


def work(case):
    op = case["op"]
    if op == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        rows = M * K + N * K + 4 * (M + N) + 2 * M * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        return dict(bytes=rows, flops=2.0 * M * N * K)
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("glr"):
        C = case["H"] * case["D"]
        n, N = case["B"] * case["T"] * C, case["seqs"] or case["B"]
        st = 4 * N * C * (2 if case["state"] else 1)
        if op == "glr_train":  # x, both gates and dy in; y and three gradients out
            return dict(bytes=8 * n * e + 2 * st + 24 * C, flops=60.0 * n)
        return dict(bytes=4 * n * e + st + 12 * C, flops=20.0 * n)
    n, r = case["T"] * case["D"], 4 if case["wide"] else e
    if op == "norm8":
        return dict(bytes=n * (e + 2 * r + 1) + 4 * case["T"] + 4 * case["D"], flops=8.0 * n)
    # x, residual, dy and dh in; y, h, and the gradients of x (its own where it differs from the residual's) and the residual out
    own_dx = e if case["p"] or r != e else 0
    return dict(bytes=n * (3 * e + 4 * r + own_dx) + 8 * case["D"], flops=20.0 * n)


def _exact_glr(s):
    """Token by token in 64 bits, all sequences side by side, and the adjoint of that loop."""
    c = s["case"]
    lens, N, C = s["lens"], len(s["lens"]), c["H"] * c["D"]
    L, dev = max(lens), s["x"].device
    place = s["seq"] * L + s["pos"]

    def lay(t):  # [B, T, H, D] -> [L, N, C], zeros behind the shorter sequences
        flat = torch.zeros(N * L, C, dtype=torch.float64, device=dev)
        flat[place] = t.reshape(-1, C).double()
        return flat.reshape(N, L, C).transpose(0, 1).contiguous()

    def unlay(t):
        return t.transpose(0, 1).reshape(N * L, C)[place].reshape(s["x"].shape)

    lam, br, bi = (s[k].double().reshape(C) for k in ("lam", "br", "bi"))
    soft = torch.logaddexp(lam, torch.zeros_like(lam))
    here = lay(torch.ones_like(s["x"], dtype=torch.float64))[..., :1]  # 0 behind a sequence's end
    rate = 1 / (1 + torch.exp(-(lay(s["r"]) + br)))
    gate = 1 / (1 + torch.exp(-(lay(s["i"]) + bi)))
    x = lay(s["x"])
    log = -POWER * soft * rate * here
    a = torch.exp(log)
    m = torch.sqrt(-torch.expm1(2 * log))
    h = s["h0"].double().reshape(N, C) if s["h0"] is not None else torch.zeros(N, C, dtype=torch.float64, device=dev)
    hs = torch.empty(L + 1, N, C, dtype=torch.float64, device=dev)
    hs[0] = h
    add = m * gate * x
    for t in range(L):
        torch.addcmul(add[t], a[t], hs[t], out=hs[t + 1])
    out = dict(y=unlay(hs[1:]), hT=hs[L].reshape(N, c["H"], c["D"]))
    if c["op"] == "glr":
        return out
    g = lay(s["dy"])
    carry = s["dhT"].double().reshape(N, C) if s["dhT"] is not None else torch.zeros_like(hs[0])
    for t in reversed(range(L)):
        g[t] += carry
        carry = a[t] * g[t]
    over = torch.where(here > 0, g / m, 0)
    dlog = (g * hs[:L] * a - over * gate * x * a * a) * here
    dr = dlog * log * (1 - rate)
    di = g * add * (1 - gate)
    shape = (c["H"], c["D"])
    out.update(dx=unlay(g * m * gate), dr=unlay(dr), di=unlay(di), dbr=dr.sum((0, 1)).reshape(shape), dbi=di.sum((0, 1)).reshape(shape),
               dlam=(-POWER / (1 + torch.exp(-lam)) * (dlog * rate).sum((0, 1))).reshape(shape))
    if s["h0"] is not None:
        out["dh0"] = carry.reshape(N, *shape)
    return out


def _exact_keep(s, T, D):
    """The dropout's factors with numbers cut into 16-bit limbs, so that no product needs more than 32 bits."""
    key, stream = (int(v) % 2 ** 64 for v in s["seed"].tolist())
    unit = torch.arange(T * D // 8, device=s["seed"].device)

    def times(word, by):
        """The upper and lower 32 bits of word * by."""
        p = [[((word >> 16 * i) & 0xFFFF) * ((by >> 16 * j) & 0xFFFF) for j in (0, 1)] for i in (0, 1)]
        mid = (p[0][0] >> 16) + (p[0][1] & 0xFFFF) + (p[1][0] & 0xFFFF)
        return p[1][1] + (p[0][1] >> 16) + (p[1][0] >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) + (p[0][0] & 0xFFFF)

    c0, c1 = unit % 2 ** 32, unit // 2 ** 32
    c2, c3 = torch.full_like(unit, stream % 2 ** 32), torch.full_like(unit, stream >> 32)
    k0, k1 = key % 2 ** 32, key >> 32
    for _ in range(7):
        hi0, lo0 = times(c0, 0xD2511F53)
        hi1, lo1 = times(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = hi1 ^ c1 ^ k0, lo1, hi0 ^ c3 ^ k1, lo0
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    bits = torch.empty(T * D // 8, 8, dtype=torch.int64, device=unit.device)
    for n, word in enumerate((c0, c1, c2, c3)):
        bits[:, 2 * n], bits[:, 2 * n + 1] = word % 65536, word // 65536
    drop = round(s["case"]["p"] * 65536)
    return (bits.reshape(T, D) >= drop).double() / (1 - drop / 65536)


def _exact_norm(s):
    c = s["case"]
    train = c["op"] == "norm_train"
    keep = _exact_keep(s, c["T"], c["D"]) if c["p"] else 1.0
    h = (s["res"].double() + keep * s["x"].double()).to(s["res"].dtype).double().requires_grad_(train)
    w = s["w"].double().requires_grad_(train)
    with torch.set_grad_enabled(train):
        y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / c["D"] + EPS) * w
    if not train:
        scale = y.abs().max(-1).values / TOP8
        return dict(y=y / scale[:, None], scale=scale, h=h)
    dn, dw = torch.autograd.grad(y, [h, w], s["dy"].double())
    dres = dn + s["dh"].double()
    return dict(y=y.detach(), h=h.detach(), dx=keep * dres, dres=dres, dw=dw)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear8":
        x, w = s["x"].double() * s["xs"].double()[:, None], s["w"].double() * s["ws"].double()[:, None]
        z = x @ w.T
        z = z if s["bias"] is None else z + s["bias"].double()
        if case["act"] == "silu":
            z = z / (1 + torch.exp(-z))
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        return dict(y=z if s["residual"] is None else z + s["residual"].double())
    if op == "glr_step":
        sr, si = (1 / (1 + torch.exp(-(s[k].double() + s[b].double()))) for k, b in (("r", "br"), ("i", "bi")))
        log = -POWER * torch.logaddexp(s["lam"].double(), torch.zeros_like(s["lam"], dtype=torch.float64)) * sr
        h = torch.exp(log) * s["h0"].double() + torch.sqrt(-torch.expm1(2 * log)) * si * s["x"].double()
        return dict(y=h, state=h)
    return _exact_glr(s) if op.startswith("glr") else _exact_norm(s)
