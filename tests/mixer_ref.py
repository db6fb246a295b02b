"""Plain 64-bit implementations of the state space mixer's operators, token by
token, and the error bounds that the kernels' roundings allow.

`U32` and `UBF` are half a step of fp32 and bf16 relative to the value.  A
result that is a sum of products is off by at most (number of roundings on
the way) * U32 times the same sum over absolute values, plus, where it is
rounded to bf16 or one operand of its products was, UBF times the value or
that sum."""
import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8


def softplus(x):
    return torch.logaddexp(x, torch.zeros_like(x))


def scan_core(q, k, v, s, a, h0):
    """One sequence: q, k [T,H,Dk] (a head each), v [T,H,Dv], step sizes s and log decays a
    [T,H], h0 [H,Dk,Dv]; (o, hT) without the skip term."""
    h, o = h0, []
    for t in range(v.shape[0]):
        h = torch.exp(a[t])[:, None, None] * h + k[t][:, :, None] * (s[t][:, None] * v[t])[:, None, :]
        o.append((q[t][:, :, None] * h).sum(1))
    return (torch.stack(o) if o else torch.zeros_like(v)), h


def scan(q, k, v, s, a, skip, h0, lens):
    """All sequences (their tokens one after another): q, k [M,G,Dk], v [M,H,Dv], h0 [N,H,Dk,Dv]."""
    R = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(R, 1), k.repeat_interleave(R, 1)
    os, hs, at = [], [], 0
    for n, ln in enumerate(lens):
        i = slice(at, at + ln)
        o, h = scan_core(q[i], k[i], v[i], s[i], a[i], h0[n])
        os.append(o)
        hs.append(h)
        at += ln
    return torch.cat(os) + skip[:, None] * v, torch.stack(hs)


def scan_with_bounds(q, k, v, dt, A, bias, skip, h0, lens, dO=None, dhT=None):
    """Results and gradients in float64, and for each the largest error that the kernels may make.

    The bounds come from the same loop over absolute values (the decays as they are), whose
    results and gradients are the sums over absolute values; a state passes about 128 roundings
    a chunk of 64 tokens (64 products, the decay, the step size, the split into three parts)."""
    N, H = len(lens), v.shape[1]
    c = 128 * ((max(lens) if lens else 0) // 64 + 2) * U32
    h0 = torch.zeros(N, H, q.shape[2], v.shape[2], dtype=torch.float64) if h0 is None else h0
    bias = torch.zeros(H, dtype=torch.float64) if bias is None else bias
    skip = torch.zeros(H, dtype=torch.float64) if skip is None else skip
    s = softplus(dt + bias)
    val, bound = {}, {}

    def both(absolute):
        f = (lambda x: x.abs()) if absolute else (lambda x: x)
        leaves = [f(q), f(k), f(v), s, s * A, f(skip), f(h0)]
        leaves = [x.clone().requires_grad_(dO is not None) for x in leaves]
        o, hT = scan(*leaves, lens)
        if dO is None:
            return o, hT, None
        gr = torch.autograd.grad([o, hT], leaves, [f(dO), f(dhT) if dhT is not None else torch.zeros_like(hT)],
                                 allow_unused=True)
        return o.detach(), hT.detach(), [torch.zeros_like(x) if g is None else g for x, g in zip(leaves, gr)]

    o, hT, gr = both(False)
    ao, ahT, ag = both(True)
    rounded = lambda x, ax: UBF * x.abs() + (UBF * (1 + 2.0 ** -6) + c) * ax  # noqa: E731
    val.update(o=o, hT=hT)
    bound.update(o=rounded(o, ao), hT=c * ahT)
    if gr is None:
        return val, bound
    dq, dk, dv, ds, da, dskip, dh0 = gr
    aq, ak, av, as_, aa, askip, ah0 = ag
    sig = torch.sigmoid(dt + bias)
    ddt, addt = (ds + A * da) * sig, (as_ + A.abs() * aa) * sig
    val.update(dq=dq, dk=dk, dv=dv, ddt=ddt, dA=(s * da).sum(0), ddt_bias=ddt.sum(0), dskip=dskip, dh0=dh0)
    bound.update(dq=rounded(dq, aq), dk=rounded(dk, ak), dv=rounded(dv, av), ddt=c * addt, dA=c * (s * aa).sum(0),
                 ddt_bias=c * addt.sum(0), dskip=c * askip, dh0=c * ah0)
    return val, bound


def conv_silu(x, w, bias, s0, lens):
    """x [M,H,D], w [H,D,W], s0 [N,W-1,H,D] -> y, sT."""
    W = w.shape[2]
    ys, ts, at = [], [], 0
    for n, ln in enumerate(lens):
        line = torch.cat([s0[n], x[at:at + ln]])
        z = bias + sum(w[:, :, j] * line[j:j + ln] for j in range(W))
        ys.append(z * torch.sigmoid(z))
        ts.append(line[ln:])
        at += ln
    return torch.cat(ys), torch.stack(ts)


def gated_norm(x, z, w, eps, gate_first):
    g = z * torch.sigmoid(z)
    u = x * g if gate_first else x
    n = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * w
    return n if gate_first else n * g


def worst(got, want, bound):
    """The largest error over its bound (where both are zero it is zero)."""
    err = (got.double().cpu() - want).abs()
    over = err / bound.clamp_min(1e-300)
    return float(torch.where(err == 0, torch.zeros_like(err), over).max()) if err.numel() else 0.0
