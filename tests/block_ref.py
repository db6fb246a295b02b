"""64-bit references of the operators around the token mixers (gated linear
recurrence, residual addition with dropout and norm, 8-bit product), written
from the definitions, with bounds on what the kernels' roundings may add.

Units: U = 2^-24 is half a step of fp32 relative to the value, and a result in
another type is off by half of its own step more (``half``)."""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def worst(got, val, bound):
    """The largest error in units of its bound; NaN counts as infinite, and equal infinities as none."""
    d = (got.double().cpu() - val).abs()
    d = torch.where(got.double().cpu() == val, torch.zeros_like(d), d)
    q = d / bound.clamp(min=1e-300)
    q = torch.where(torch.isnan(q), torch.full_like(q, torch.inf), q)
    return float(q.max()) if q.numel() else 0.0


# ------------------------------------------------ the gated linear recurrence


def glr(x, r, i, lam, br, bi, h0, lens, power, dy=None, dhT=None, dtype=torch.float64):
    """Token by token over rows [R, C] of sequences of these lengths: (values, bounds) of y, hT and, given dy,
    of all gradients.  `dtype`: that of y, dx, dr, di.  Everything comes in as float64; br, bi, h0, dhT may be None.

    Bounds.  sigmoid(z) is off by its argument's rounding, 2 |z| U, and a few operations: cs = 4 + 3 |z| units.  log a
    has cs + 4 of them, so that a has ca = |log a| (cs + 4) + 3; 1 - a^2 has at most those of log a and a few, its
    root half: cm = cs / 2 + 6.  A state's error is its predecessor's times a, plus what a and the input add; the
    products over tiles have one more rounding a token, counted in ca."""
    R, C = x.shape
    N = len(lens)
    z0 = torch.zeros(C, dtype=torch.float64)
    br_, bi_ = z0 if br is None else br, z0 if bi is None else bi
    soft = torch.logaddexp(lam, z0)
    s, si = torch.sigmoid(r + br_), torch.sigmoid(i + bi_)
    l = -power * soft * s
    a = torch.exp(l)
    m = torch.sqrt(-torch.expm1(2 * l))
    u = si * x
    csr = 4 + 3 * (r.abs() + br_.abs()).clamp(max=200)
    csi = 4 + 3 * (i.abs() + bi_.abs()).clamp(max=200)
    ca = l.abs() * (csr + 4) + 3
    cb = csr / 2 + csi + 10
    y, Eh, Habs, before, Ebefore = (torch.zeros(R, C, dtype=torch.float64) for _ in range(5))
    hT, EhT = torch.zeros(N, C, dtype=torch.float64), torch.zeros(N, C, dtype=torch.float64)
    at = 0
    for n, ln in enumerate(lens):
        h = z0.clone() if h0 is None else h0[n].clone()
        e, ab = torch.zeros_like(h), h.abs()
        for t in range(at, at + ln):
            before[t], Ebefore[t] = h, e
            b = m[t] * u[t]
            e = a[t] * e + U * (ca[t] * a[t] * ab + cb[t] * b.abs())
            ab = a[t] * ab + b.abs()
            h = a[t] * h + b
            y[t], Eh[t], Habs[t] = h, e, ab
        hT[n], EhT[n] = h, e
        at += ln
    # results below the fp32 range come out as zeros; a decay below 2^-126 does too, and what it multiplies is lost
    # whole: at power 1e4 a = 1.154e-38 < 2^-126 = 1.175e-38, log a = -87.4, and dr loses g log a a h_{t-1} = 1.23e-37
    tiny, flush = 1e-37, 2.0 ** -126
    val = dict(y=y, hT=hT)
    bound = dict(y=Eh * (1 + half(dtype)) + half(dtype) * y.abs() + tiny, hT=EhT + tiny)
    if dy is None:
        return val, bound
    g, Eg, Gabs = (torch.zeros(R, C, dtype=torch.float64) for _ in range(3))
    dh0, Edh0 = torch.zeros(N, C, dtype=torch.float64), torch.zeros(N, C, dtype=torch.float64)
    at = R_used = sum(lens)
    for n in reversed(range(N)):
        c = z0.clone() if dhT is None else dhT[n].clone()
        e, ab = torch.zeros_like(c), c.abs()
        for t in range(at - 1, at - lens[n] - 1, -1):
            g[t] = dy[t] + c
            Gabs[t] = dy[t].abs() + ab
            Eg[t] = e + U * Gabs[t]
            e = a[t] * Eg[t] + U * ca[t] * a[t] * Gabs[t]
            c, ab = a[t] * g[t], a[t] * Gabs[t]
        dh0[n], Edh0[n] = c, e
        at -= lens[n]
    over = torch.where(m > 0, l / m.clamp(min=1e-300), torch.zeros_like(m))  # log a / m, 0 where a = 1
    t1, t2 = l * a * before, u * a * a * over
    W = g * (t1 - t2)
    EW = (t1.abs() + t2.abs()) * Eg + (g * l * a).abs() * Ebefore + U * Gabs * (
        t1.abs() * (ca + csr + 8) + t2.abs() * (2 * ca + 1.5 * csr + csi + 20)) + flush * Gabs * l.abs() * before.abs()
    dr = (1 - s) * W
    Edr = (1 - s) * EW + 3 * U * W.abs()  # 1 - s has the absolute error of s
    dx = g * m * si
    Edx = m * si * (Eg + U * Gabs * (csr / 2 + csi + 12))
    di = g * m * u * (1 - si)
    Edi = (m * u).abs() * ((1 - si) * (Eg + U * Gabs * (csr / 2 + csi + 12)) + 3 * U * Gabs * (1 + csi * si * (1 - si)))
    Edr = Edr + U * csr * s * (1 - s) * W.abs()
    live = slice(0, R_used)
    adds = (R_used // 16 + 100) * U  # a thread's rows, the threads, the segments
    ratio = torch.sigmoid(lam) / soft
    val.update(dx=dx, dr=dr, di=di, dlam=ratio * W[live].sum(0), dbr=dr[live].sum(0), dbi=di[live].sum(0), dh0=dh0)
    rnd = lambda e, v: e * (1 + half(dtype)) + half(dtype) * v.abs() + tiny  # noqa: E731
    total = lambda e, v: e[live].sum(0) + adds * v[live].abs().sum(0) + tiny  # noqa: E731
    bound.update(dx=rnd(Edx, dx), dr=rnd(Edr, dr), di=rnd(Edi, di), dlam=ratio * (total(EW, W) + 12 * U * W[live].sum(0).abs()),
                 dbr=total(Edr, dr), dbi=total(Edi, di), dh0=Edh0 + tiny)
    for k in ("y", "dx", "dr", "di"):
        val[k][R_used:] = 0
    return val, bound


# --------------------------------------- residual addition, dropout and norm


def philox(key, stream, block):
    """Philox4x32 with 7 rounds on Python's integers: four words."""
    c = [block & 0xFFFFFFFF, block >> 32, stream & 0xFFFFFFFF, stream >> 32]
    k = [key & 0xFFFFFFFF, key >> 32]
    for _ in range(7):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_factors(seed, p, rows, D, row0=0):
    """The dropout's factors [rows, D] in float64, from row `row0` on."""
    drop = round(p * 65536)
    if not drop:
        return torch.ones(rows, D, dtype=torch.float64)
    key, stream = (int(v) % 2 ** 64 for v in seed)
    out = torch.empty(rows, D // 8, 8, dtype=torch.float64)
    for i in range(rows):
        for b in range(D // 8):
            words = philox(key, stream, (row0 + i) * D // 8 + b)
            bits = [w >> s & 0xFFFF for w in words for s in (0, 16)]
            out[i, b] = torch.tensor([float(v >= drop) for v in bits], dtype=torch.float64)
    return out.reshape(rows, D) * (65536.0 / (65536 - drop))


def norm(h, w, eps, dy=None, dh=None):
    """n = h / rms, y = n w and, given dy, the gradients of h and w; float64 rows [R, D], w None: y = h."""
    if w is None:
        return h
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = h * r
    if dy is None:
        return n * w
    dn = dy * w
    dres = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return n * w, dres if dh is None else dres + dh, (dy * n).sum(0)


def norm_bounds(h, w, eps, dtype, res_dtype, dy, dh, keep):
    """Bounds of y, dres, dx, dw.  A row's sum is a lane's up to 32 values and a tree over 256: 48 U at most, half of it
    for the root; products and the root a few more: 32 U in all for n.  dn's mean carries the absolute terms."""
    D = h.shape[-1]
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n, dn = h * r, dy * w
    y, dres, dw = norm(h, w, eps, dy, dh)
    Edres = U * (40 * r * dn.abs() + 120 * r * n.abs() * (dn * n).abs().mean(-1, keepdim=True) + dres.abs() * 2
                 + (0 if dh is None else dh.abs()))
    rows = h.shape[0]
    return dict(y=(half(dtype) + 36 * U) * y.abs() + 1e-37, dres=Edres + half(res_dtype) * dres.abs() + 1e-37,
                dx=keep * (Edres + (half(dtype) + 2 * U) * dres.abs()) + 1e-37,
                dw=((rows // 256 + 1100) * U + 34 * U) * (dy * n).abs().sum(0) + 1e-37)


# ----------------------------------------------------------- 8-bit product


def linear8(x, xs, w, ws, bias, residual, act):
    """float64 y, and a bound: half a step of bf16, fp32's few roundings, and what the matrix instructions cut.  These
    align eight neighbouring products to the largest one and cut, towards zero, what lies 13 bits below its power of
    two (test_gpu_linear8.py shows it), and add the eight to an fp32 sum.  So a group of eight is off by at most B = 7
    x 2^-13 of its largest product, itself at most the product of the group's largest |x| and |w|.  The cuts take the
    products' signs, which are as often one as the other: by Hoeffding's inequality groups that are independent are
    off by 7.5 sqrt(sum B^2) together with a probability of 2 e^-28 at most."""
    p = x @ w.t()
    z = p * xs[:, None] * ws + (0 if bias is None else bias)
    y = z * torch.sigmoid(z) if act == "silu" else z * torch.special.ndtr(z) if act == "gelu" else z
    y = y if residual is None else y + residual
    most = lambda t: t.abs().reshape(t.shape[0], -1, 8).amax(-1)  # noqa: E731
    cut = 7 * 2.0 ** -13 * torch.minimum(most(x) @ most(w).t(), 7.5 * torch.sqrt(most(x) ** 2 @ (most(w) ** 2).t()))
    Ez = (cut + U * (x.shape[1] // 8 + 2) * (x.abs() @ w.abs().t())) * xs[:, None].abs() * ws.abs() + 4 * U * (
        z.abs() + (0 if bias is None else bias.abs()))
    # the activations' slope is at most 1.13, and their own error a few units of z
    return y, half(torch.bfloat16) * y.abs() + 1.2 * Ez + 24 * U * z.abs() * (1 + z.abs()) + 1e-37
