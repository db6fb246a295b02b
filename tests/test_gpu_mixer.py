"""GPU parity of the state space mixer's operators (scan, stateful short
convolution, gated norm) with the 64-bit reference, within the bounds that
their roundings allow, and the ways a program uses them: continued prompts,
single tokens, streams, graphs, autograd, the three together."""
import ctypes

import pytest
import torch

import chunkwise_delta_rule_wy_amd as dn
import mixer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def randn(*shape, seed=0, scale=1.0, dtype=F32):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def cu_of(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def scan_inputs(B, T, H, G, dk, dv, lens=None, state=True, seed=0, A=None, dtype=BF):
    N = len(lens) if lens else B
    silu = torch.nn.functional.silu
    x = dict(q=silu(randn(B, T, G, dk, seed=seed)).to(dtype), k=silu(randn(B, T, G, dk, seed=seed + 1)).to(dtype),
             v=silu(randn(B, T, H, dv, seed=seed + 2)).to(dtype), dt=randn(B, T, H, seed=seed + 3),
             A=-1 - 15 * torch.rand(H, generator=torch.Generator().manual_seed(seed + 4)) if A is None
             else torch.full((H,), A),
             dt_bias=randn(H, seed=seed + 5) - 3, skip=randn(H, seed=seed + 6),
             h0=randn(N, H, dk, dv, seed=seed + 7, scale=0.3) if state else None)
    dO = randn(B, T, H, dv, seed=seed + 8).to(dtype)
    dhT = randn(N, H, dk, dv, seed=seed + 9, scale=0.3) if state else None
    return x, dO, dhT, lens or [T] * B


def cuda(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def reference(x, lens, dO=None, dhT=None):
    f = lambda t: None if t is None else t.double()  # noqa: E731
    flat = lambda t: None if t is None else t.double().flatten(0, 1)  # noqa: E731
    return ref.scan_with_bounds(flat(x["q"]), flat(x["k"]), flat(x["v"]), flat(x["dt"]), f(x["A"]), f(x["dt_bias"]),
                                f(x["skip"]), f(x["h0"]), lens, flat(dO), f(dhT))


def check(got, val, bound, names):
    for n in names:
        g = got[n].reshape(val[n].shape)
        assert torch.isfinite(g).all(), n
        assert ref.worst(g, val[n], bound[n]) <= 1, (n, ref.worst(g, val[n], bound[n]))


SHAPES = [
    # B, T, H, G, dk, dv, packed lengths, carried state
    (1, 1, 1, 1, 64, 64, None, True),
    (2, 3, 2, 1, 128, 64, None, False),
    (1, 63, 2, 2, 64, 128, None, True),
    (2, 64, 4, 2, 128, 64, None, True),
    (1, 65, 3, 1, 64, 192, None, True),
    (3, 130, 4, 1, 128, 128, None, False),
    (1, 577, 2, 1, 128, 64, None, True),
    (2, 512, 1, 1, 64, 64, None, True),
    (1, 2117, 2, 1, 64, 64, None, True),   # more than 32 chunks and few streams: cut into segments
    (1, 2112, 1, 1, 128, 64, None, False),
    (1, 2300, 2, 2, 64, 64, [0, 2200, 37, 0, 63, 0], True),
    (1, 300, 4, 2, 64, 64, [0, 1, 63, 64, 0, 65, 107, 0], True),
    (1, 700, 2, 1, 128, 128, [1, 1, 600, 98], False),
    (1, 5, 6, 3, 64, 64, [0, 0, 5], True),
]


@pytest.mark.parametrize("B,T,H,G,dk,dv,lens,state", SHAPES)
def test_scan_and_gradients(B, T, H, G, dk, dv, lens, state):
    x, dO, dhT, ls = scan_inputs(B, T, H, G, dk, dv, lens, state)
    val, bound = reference(x, ls, dO, dhT)
    d = cuda(x)
    cu = cu_of(lens) if lens else None
    o, hT = dn.ssm_fwd(**d, cu_seqlens=cu)
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], dO.cuda(),
                    None if dhT is None else dhT.cuda(), cu)
    torch.cuda.synchronize()
    assert o.dtype == gr["dq"].dtype == gr["dk"].dtype == gr["dv"].dtype == BF
    check(dict(gr, o=o, hT=hT), val, bound, list(val))


@pytest.mark.parametrize("B,T,H,G,dk,dv", [(256, 2, 12, 1, 64, 64), (130, 3, 22, 2, 128, 64), (86, 65, 9, 3, 64, 64)])
def test_scan_many_heads_of_a_key(B, T, H, G, dk, dv):
    # chunks enough that one workgroup passes through all heads of a group, eight at a time
    x, dO, dhT, ls = scan_inputs(B, T, H, G, dk, dv, state=T < 60)
    val, bound = reference(x, ls, dO, dhT)
    d = cuda(x)
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], dO.cuda(),
                    None if dhT is None else dhT.cuda())
    check(gr, val, bound, [n for n in gr if n in val])


@pytest.mark.parametrize("A,shift", [(0.0, 0.0), (-1e-4, 0.0), (-40.0, 3.0), (-1.0, -30.0), (-2000.0, 5.0)])
def test_scan_extreme_decays(A, shift):
    # no decay, hardly any, one token's memory, vanishing steps, decays that underflow at once
    x, dO, dhT, ls = scan_inputs(1, 150, 2, 1, 64, 64, A=A)
    x["dt_bias"] = torch.full((2,), shift)
    val, bound = reference(x, ls, dO, dhT)
    d = cuda(x)
    o, hT = dn.ssm_fwd(**d)
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], dO.cuda(), dhT.cuda())
    # results below the fp32 range come out as zeros
    bound = {k: b + 1e-37 for k, b in bound.items()}
    check(dict(gr, o=o, hT=hT), val, bound, list(val))


def test_scan_without_optional_parameters():
    x, dO, _, ls = scan_inputs(1, 70, 2, 2, 64, 64, state=False)
    x["dt_bias"] = x["skip"] = None
    val, bound = reference(x, ls, dO)
    d = cuda(x)
    o, hT = dn.ssm_fwd(**d, output_final_state=False)
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], None, None, None, dO.cuda())
    assert hT is None and gr["ddt_bias"] is None and gr["dskip"] is None
    check(dict(gr, o=o), val, bound, ["o", "dq", "dk", "dv", "ddt", "dA"])


def test_scan_of_no_tokens_passes_states():
    x, _, dhT, _ = scan_inputs(2, 0, 2, 1, 64, 64)
    d = cuda(x)
    o, hT = dn.ssm_fwd(**d)
    assert o.shape == (2, 0, 2, 64) and torch.equal(hT, d["h0"])
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], d["v"], dhT.cuda())
    assert torch.equal(gr["dh0"].cpu(), dhT)
    assert not gr["dA"].any() and not gr["ddt_bias"].any() and not gr["dskip"].any()


def test_scan_continues_in_pieces():
    # pieces carried by hT: the second within the bound of the whole
    x, _, _, ls = scan_inputs(2, 200, 4, 2, 128, 64)
    val, bound = reference(x, ls)
    d = cuda(x)
    h, outs = d["h0"], []
    for a, b in ((0, 70), (70, 71), (71, 200)):
        part = {k: d[k][:, a:b].contiguous() for k in ("q", "k", "v", "dt")}
        o, h = dn.ssm_fwd(**part, A=d["A"], dt_bias=d["dt_bias"], skip=d["skip"], h0=h)
        outs.append(o)
    check(dict(o=torch.cat(outs, 1), hT=h), val, bound, ["o", "hT"])


@pytest.mark.parametrize("dtype,dk,dv,H,G", [(BF, 64, 64, 4, 2), (F32, 64, 64, 2, 1), (BF, 128, 128, 2, 2),
                                            (F32, 128, 192, 3, 1), (BF, 64, 256, 1, 1)])
def test_scan_step_by_step(dtype, dk, dv, H, G):
    B, T = 3, 5
    x, _, _, ls = scan_inputs(B, T, H, G, dk, dv, dtype=dtype)
    val, _ = reference(x, ls)
    # a step: Dk products and as many sums, the decay and the step size (about 16 roundings)
    c = (dk + 16) * (T + 1) * ref.U32
    big, _ = reference({k: v.abs() if k in ("q", "k", "v", "skip", "h0") else v for k, v in x.items()}, ls)
    d = cuda(x)
    state, outs = d["h0"].clone(), []
    for t in range(T):
        outs.append(dn.ssm_step(d["q"][:, t].contiguous(), d["k"][:, t].contiguous(), d["v"][:, t].contiguous(),
                                d["dt"][:, t].contiguous(), d["A"], d["dt_bias"], d["skip"], state))
    bound = dict(o=c * big["o"] + (ref.UBF * val["o"].abs() if dtype == BF else 0), hT=c * big["hT"])
    check(dict(o=torch.stack(outs, 1), hT=state), val, bound, ["o", "hT"])


def test_scan_sequences_do_not_touch():
    # a value that is not finite in one packed sequence leaves the others as they are
    lens = [70, 64, 130]
    x, dO, dhT, _ = scan_inputs(1, 264, 4, 2, 64, 64, lens)
    d, cu = cuda(x), cu_of(lens)
    o, hT = dn.ssm_fwd(**d, cu_seqlens=cu)
    bad = dict(d, v=d["v"].clone())
    bad["v"][0, 100, 1, 3] = float("nan")
    bad["v"][0, 70, 0, 0] = float("inf")
    o2, hT2 = dn.ssm_fwd(**bad, cu_seqlens=cu)
    assert torch.equal(o2[:, :70], o[:, :70]) and torch.equal(o2[:, 134:], o[:, 134:])
    assert torch.equal(hT2[0], hT[0]) and torch.equal(hT2[2], hT[2]) and not torch.isfinite(hT2[1]).all()


def test_scan_repeats_bit_for_bit():
    x, dO, dhT, _ = scan_inputs(2, 700, 4, 1, 128, 64)
    d = cuda(x)
    args = (d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"])
    o, hT = dn.ssm_fwd(*args)
    gr = dn.ssm_bwd(*args, dO.cuda(), dhT.cuda())
    for _ in range(4):
        o2, h2 = dn.ssm_fwd(*args)
        g2 = dn.ssm_bwd(*args, dO.cuda(), dhT.cuda())
        assert torch.equal(o, o2) and torch.equal(hT, h2)
        assert all(torch.equal(gr[n], g2[n]) for n in gr)


@pytest.mark.parametrize("B,T,H,G,dk,dv,lens", [
    (4, 4096, 32, 1, 128, 64, None), (1, 16384, 16, 4, 64, 128, None), (2, 4096, 5, 5, 128, 192, None),
    (1, 20000, 16, 2, 128, 128, [9000, 1, 64, 10000, 935])])
def test_scan_repeats_at_full_size(B, T, H, G, dk, dv, lens):
    """A matrix result read too early, or a missing barrier, shows as values that change between
    runs of a full device."""
    torch.manual_seed(7)
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    args = (r(B, T, G, dk).to(BF), r(B, T, G, dk).to(BF), r(B, T, H, dv).to(BF), r(B, T, H) - 3, -4 * torch.rand(H).cuda(),
            r(H), r(H), r(len(lens) if lens else B, H, dk, dv))
    dO, dhT, cu = r(B, T, H, dv).to(BF), torch.randn_like(args[-1]), cu_of(lens) if lens else None
    first = None
    for _ in range(8):
        o, hT = dn.ssm_fwd(*args, cu)
        out = dict(dn.ssm_bwd(*args, dO, dhT, cu), o=o, hT=hT)
        first = first or out
        for n in out:
            assert torch.equal(out[n], first[n]), n
    assert all(torch.isfinite(t).all() for t in first.values())


# ------------------------------------------------------------ convolution

CONVS = [
    # B, T, H, D, W, packed lengths, carried state, bias
    (1, 1, 1, 8, 4, None, True, True), (2, 2, 3, 16, 4, None, True, True), (2, 37, 2, 40, 3, None, False, True),
    (1, 100, 5, 128, 4, None, True, False), (3, 70, 1, 8, 1, None, False, True), (1, 300, 9, 64, 2, None, True, True),
    (1, 90, 2, 24, 4, [0, 1, 2, 3, 4, 0, 31, 49, 0], True, True), (1, 40, 1, 520, 4, [33, 7], False, False),
    (1, 9000, 1, 16, 4, None, True, True),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,D,W,lens,state,bias", CONVS)
def test_conv_silu_and_gradients(B, T, H, D, W, lens, state, bias, dtype):
    ls = lens or [T] * B
    N = len(ls)
    x, w = randn(B, T, H, D, seed=1, dtype=dtype), randn(H, D, W, seed=2, scale=0.5)
    b = randn(H, D, seed=3) if bias else None
    s0 = randn(N, W - 1, H, D, seed=4, dtype=dtype) if state else None
    dy, dsT = randn(B, T, H, D, seed=5, dtype=dtype), randn(N, W - 1, H, D, seed=6, dtype=dtype) if state else None
    z0 = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    leaves = [x.double().reshape(-1, H, D), w.double(), b.double() if bias else z0(H, D),
              s0.double() if state else z0(N, W - 1, H, D)]
    leaves = [t.requires_grad_() for t in leaves]
    y, sT = ref.conv_silu(*leaves, ls)
    up = [dy.double().reshape(-1, H, D), dsT.double() if state else torch.zeros_like(sT)]
    gx, gw, gb, gs = torch.autograd.grad([y, sT], leaves, up)
    # sums over absolute values: |z| and, as |silu'| < 1.1, |dz| <= 1.1 |dy|
    al = [t.detach().abs() for t in leaves]
    za, _ = ref.conv_silu(al[0], al[1], al[2], al[3], ls)  # silu(z) >= z - 0.28 for z >= 0
    za = za + 0.28
    u = (W + 16) * ref.U32
    r = ref.UBF if dtype == BF else 2 * ref.U32
    # dz from z: silu'' is below 0.5, so an error of z reaches dz by half
    dza = (1.1 + 0.5 * za) * up[0].abs()
    ga = [t.clone().requires_grad_() for t in (al[0], al[1], al[2], al[3])]
    lin, last = [], []
    at = 0
    for n, ln in enumerate(ls):
        line = torch.cat([ga[3][n], ga[0][at:at + ln]])
        lin.append(ga[2] + sum(ga[1][:, :, j] * line[j:j + ln] for j in range(W)))
        last.append(line[ln:])
        at += ln
    ax, aw, ab, as_ = torch.autograd.grad([torch.cat(lin), torch.stack(last)], ga, [dza, up[1].abs()])
    c = (T * B + 64) * ref.U32  # the weights' gradients are sums over all tokens
    val = dict(y=y, sT=sT, dx=gx, dw=gw, dbias=gb, ds0=gs)
    bound = dict(y=r * y.abs() + u * (za + 1), sT=torch.zeros_like(sT), dx=r * gx.abs() + u * ax, dw=(c + u) * aw,
                 dbias=(c + u) * ab, ds0=r * gs.abs() + u * as_)
    c_ = lambda t: None if t is None else t.cuda()  # noqa: E731
    cu = cu_of(lens) if lens else None
    yg, sg = dn.conv_silu(x.cuda(), w.cuda(), c_(b), c_(s0), cu)
    gr = dn.conv_silu_bwd(x.cuda(), w.cuda(), c_(b), c_(s0), dy.cuda(), c_(dsT), cu)
    assert (gr["dbias"] is None) == (not bias)
    names = [n for n in val if n != "dbias" or bias]
    check(dict(gr, y=yg, sT=sg), {k: v.detach() for k, v in val.items()}, {k: v.detach() for k, v in bound.items()}, names)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_conv_silu_step_equals_prompt(W, dtype):
    B, T, H, D = 3, 7, 2, 24
    x, w, b = randn(B, T, H, D, seed=1, dtype=dtype).cuda(), randn(H, D, W, seed=2).cuda(), randn(H, D, seed=3).cuda()
    s0 = randn(B, W - 1, H, D, seed=4, dtype=dtype).cuda()
    y, sT = dn.conv_silu(x, w, b, s0)
    state = s0.clone()
    for t in range(T):
        assert torch.equal(dn.conv_silu_step(x[:, t].contiguous(), w, b, state), y[:, t])
    assert torch.equal(state, sT)


def test_conv_silu_extreme_values():
    # z far from zero in both directions: silu is 0 or z, its slope 0 or 1
    x = torch.tensor([-3e38, -1e4, -100.0, 0.0, 100.0, 1e4, 3e38, 1.0]).reshape(1, 1, 1, 8).cuda()
    w = torch.ones(1, 8, 1).cuda()
    y, _ = dn.conv_silu(x, w)
    gr = dn.conv_silu_bwd(x, w, None, None, torch.ones_like(x))
    want = x * (x > 0)
    assert torch.equal(y[..., [0, 1, 3, 4, 5, 6]], want[..., [0, 1, 3, 4, 5, 6]]) and y[0, 0, 0, 2].abs() < 1e-40
    assert torch.isfinite(gr["dx"]).all() and torch.equal(gr["dx"].flatten()[[1, 3, 4, 5]].cpu(), torch.tensor([0, .5, 1, 1]))


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("shape,heads", [((1, 1, 1, 8), False), ((2, 3, 5, 64), True), ((2, 9, 4, 128), False),
                                         ((70, 3, 72), True), ((5, 256), False), ((1, 40, 2, 520), True),
                                         ((3, 1000), False), ((2, 5, 2, 2048), True), ((9, 4104), False),
                                         ((2, 2, 8192), True), ((1500, 2, 64), True)])
def test_gated_norm_and_gradients(shape, heads, first, dtype):
    D, eps = shape[-1], 1e-5
    x, z, dy = (randn(*shape, seed=i, dtype=dtype) for i in (1, 2, 3))
    w = randn(*(shape[-2:] if heads else (D,)), seed=4)
    leaves = [t.double().requires_grad_() for t in (x, z, w)]
    y = ref.gated_norm(*leaves, eps, first)
    gx, gz, gw = torch.autograd.grad(y, leaves, dy.double())
    X, Z, Wd, DY = leaves[0].detach(), leaves[1].detach(), w.double(), dy.double()
    sg = torch.sigmoid(Z)
    gate, slope = (Z * sg).abs(), (sg * (1 + Z * (1 - sg))).abs()
    U = X.abs() * gate if first else X.abs()
    r = 1 / torch.sqrt((U * U).mean(-1, keepdim=True) + eps)
    n = U * r
    dnn = DY.abs() * Wd.abs() * (1 if first else gate)
    du = r * (dnn + n * (dnn * n).mean(-1, keepdim=True))
    # a mean of D products, the root, the gate: about D + 32 roundings
    c = (D + 32) * ref.U32
    rnd = ref.UBF if dtype == BF else 2 * ref.U32
    ax, az = (du * gate, du * X.abs() * (slope + ref.U32)) if first else (du, DY.abs() * Wd.abs() * n * (slope + ref.U32))
    aw = DY.abs() * n * (1 if first else gate)
    aw = aw.reshape(-1, *w.shape).sum(0)
    rows = x.numel() // w.numel()
    val = dict(y=y.detach(), dx=gx, dz=gz, dw=gw)
    # the slope's own terms, z (1 - sigmoid), may cancel: their size is below 1.3
    bound = dict(y=rnd * y.detach().abs() + c * n * Wd.abs() * (1 if first else gate), dx=rnd * gx.abs() + c * ax,
                 dz=rnd * gz.abs() + c * (az + (du * X.abs() if first else DY.abs() * Wd.abs() * n) * 1.3),
                 dw=(c + rows * ref.U32) * aw)
    yg = dn.gated_norm(x.cuda(), z.cuda(), w.cuda(), eps, first)
    dx, dz, dw = dn.gated_norm_bwd(x.cuda(), z.cuda(), w.cuda(), dy.cuda(), eps, first)
    check(dict(y=yg, dx=dx, dz=dz, dw=dw), val, bound, list(val))


def test_gated_norm_zero_rows_and_no_rows():
    x, z, w = torch.zeros(3, 64).cuda(), randn(3, 64, seed=1).cuda(), torch.ones(64).cuda()
    assert not dn.gated_norm(x, z, w).any()
    for g in dn.gated_norm_bwd(x, z, w, x):
        assert not g.any()
    e = torch.zeros(0, 2, 64).cuda()
    assert dn.gated_norm(e, e, w).shape == e.shape
    assert not dn.gated_norm_bwd(e, e, w, e)[2].any()


# ------------------------------------------------------------- in programs

def mixer_weights(H, G, dk, dv, W):
    return cuda(dict(wv=randn(H, dv, W, seed=31, scale=0.5), bv=randn(H, dv, seed=32), wq=randn(G, dk, W, seed=33, scale=0.5),
                     wk=randn(G, dk, W, seed=34, scale=0.5), A=-1 - randn(H, seed=35).abs(), dt_bias=randn(H, seed=36) - 3,
                     skip=randn(H, seed=37), wn=randn(dv, seed=38)))


def test_mixer_prompt_then_tokens():
    """Convolutions, scan and norm over a prompt, continued token by token from the carried
    states, against the same operators over the whole sequence."""
    B, T, P, H, G, dk, dv, W = 2, 90, 83, 4, 2, 64, 64, 4
    p = mixer_weights(H, G, dk, dv, W)
    xv, xq, xk, z = (randn(B, T, *s, seed=i, dtype=BF).cuda()
                     for i, s in ((1, (H, dv)), (2, (G, dk)), (3, (G, dk)), (4, (H, dv))))
    dt = randn(B, T, H, seed=5).cuda()

    def prompt(a, b, sv=None, sq=None, sk=None, h=None):
        cut = lambda t: t[:, a:b].contiguous()  # noqa: E731
        v, sv = dn.conv_silu(cut(xv), p["wv"], p["bv"], sv)
        q, sq = dn.conv_silu(cut(xq), p["wq"], None, sq)
        k, sk = dn.conv_silu(cut(xk), p["wk"], None, sk)
        o, h = dn.ssm_fwd(q, k, v, cut(dt), p["A"], p["dt_bias"], p["skip"], h)
        return o, dn.gated_norm(o, cut(z), p["wn"]), sv, sq, sk, h

    o_all, y_all, *_, h_all = prompt(0, T)
    o, y, sv, sq, sk, h = prompt(0, P)
    # the same chunks, the same arithmetic, up to the chunk the prompt ends in
    assert torch.equal(o[:, :64], o_all[:, :64]) and torch.equal(y[:, :64], y_all[:, :64])
    outs = []
    for t in range(P, T):
        tok = lambda s: s[:, t].contiguous()  # noqa: E731
        v = dn.conv_silu_step(tok(xv), p["wv"], p["bv"], sv)
        q = dn.conv_silu_step(tok(xq), p["wq"], None, sq)
        k = dn.conv_silu_step(tok(xk), p["wk"], None, sk)
        o = dn.ssm_step(q, k, v, tok(dt), p["A"], p["dt_bias"], p["skip"], h)
        outs.append((o, dn.gated_norm(o, tok(z), p["wn"])))
    # the convolved q, k, v are the same bits either way, so both are within their bounds of one value
    v, _ = dn.conv_silu(xv, p["wv"], p["bv"])
    q, _ = dn.conv_silu(xq, p["wq"])
    k, _ = dn.conv_silu(xk, p["wk"])
    x = dict(q=q, k=k, v=v, dt=dt, A=p["A"], dt_bias=p["dt_bias"], skip=p["skip"], h0=None)
    val, bound = reference({n: None if t is None else t.cpu() for n, t in x.items()}, [T] * B)
    o_steps = torch.cat([o_all[:, :P], torch.stack([a for a, _ in outs], 1)], 1)
    check(dict(o=o_steps, hT=h), val, bound, ["o", "hT"])
    check(dict(o=o_all, hT=h_all), val, bound, ["o", "hT"])
    # and the norm of a token is the norm of the row
    assert torch.equal(torch.stack([b for _, b in outs], 1),
                       dn.gated_norm(torch.stack([a for a, _ in outs], 1), z[:, P:].contiguous(), p["wn"]))


def mixer_loss(p, xv, xq, xk, dt, z, cu, weight):
    v, _ = dn.conv_silu_fn(xv, p["wv"], p["bv"], None, cu)
    q, _ = dn.conv_silu_fn(xq, p["wq"], None, None, cu)
    k, _ = dn.conv_silu_fn(xk, p["wk"], None, None, cu)
    o, _ = dn.ssm_scan(q, k, v, dt, p["A"], p["dt_bias"], p["skip"], None, cu)
    return (dn.gated_norm_fn(o, z, p["wn"]).float() * weight).sum()


def test_mixer_trains_through_autograd():
    T, H, G, dk, dv, lens = 150, 4, 2, 64, 64, [40, 0, 110]
    cu = cu_of(lens)
    p = {n: t.requires_grad_() for n, t in mixer_weights(H, G, dk, dv, 4).items()}
    xv, xq, xk, z = (randn(1, T, *s, seed=i, dtype=BF).cuda().requires_grad_()
                     for i, s in ((1, (H, dv)), (2, (G, dk)), (3, (G, dk)), (4, (H, dv))))
    dt, wt = randn(1, T, H, seed=5).cuda().requires_grad_(), randn(1, T, H, dv, seed=6).cuda()
    mixer_loss(p, xv, xq, xk, dt, z, cu, wt).backward()
    # the chain by hand, from the same operators
    with torch.no_grad():
        v, _ = dn.conv_silu(xv, p["wv"], p["bv"], None, cu)
        q, _ = dn.conv_silu(xq, p["wq"], None, None, cu)
        k, _ = dn.conv_silu(xk, p["wk"], None, None, cu)
        args = (q, k, v, dt, p["A"], p["dt_bias"], p["skip"], None)
        o, _ = dn.ssm_fwd(*args, cu)
        do, dz, dwn = dn.gated_norm_bwd(o, z, p["wn"], wt.to(BF))
        g = dn.ssm_bwd(*args, do, None, cu)
        gv = dn.conv_silu_bwd(xv, p["wv"], p["bv"], None, g["dv"], None, cu)
        gq = dn.conv_silu_bwd(xq, p["wq"], None, None, g["dq"], None, cu)
        gk = dn.conv_silu_bwd(xk, p["wk"], None, None, g["dk"], None, cu)
    for a, b in ((xv.grad, gv["dx"]), (xq.grad, gq["dx"]), (xk.grad, gk["dx"]), (z.grad, dz), (dt.grad, g["ddt"]),
                 (p["wv"].grad, gv["dw"]), (p["bv"].grad, gv["dbias"]), (p["wq"].grad, gq["dw"]), (p["wn"].grad, dwn),
                 (p["wk"].grad, gk["dw"]), (p["A"].grad, g["dA"]), (p["dt_bias"].grad, g["ddt_bias"]),
                 (p["skip"].grad, g["dskip"])):
        assert torch.equal(a, b)


def test_gradients_of_states_through_autograd():
    # only the final states are used: dO and dy are absent
    x, _, dhT, ls = scan_inputs(1, 70, 2, 1, 64, 64)
    val, bound = reference(x, ls, torch.zeros(1, 70, 2, 64), dhT)
    d = {k: t.requires_grad_() for k, t in cuda(x).items()}
    _, hT = dn.ssm_scan(**d)
    hT.backward(dhT.cuda())
    got = dict(dq=d["q"].grad, dk=d["k"].grad, dv=d["v"].grad, ddt=d["dt"].grad, dA=d["A"].grad, dh0=d["h0"].grad)
    check(got, val, bound, list(got))
    xc = randn(1, 2, 1, 8, seed=1).cuda().requires_grad_()
    s0 = randn(1, 3, 1, 8, seed=2).cuda().requires_grad_()
    _, sT = dn.conv_silu_fn(xc, torch.ones(1, 8, 4).cuda(), None, s0)
    up = randn(1, 3, 1, 8, seed=3).cuda()
    sT.backward(up)
    assert torch.equal(xc.grad[0], up[0, 1:]) and torch.equal(s0.grad[0, 2], up[0, 0]) and not s0.grad[0, :2].any()


def test_gradients_that_start_between_units():
    # torch.cat hands its parts slices of one gradient, here an odd number of elements in
    x, _, _, _ = scan_inputs(1, 70, 2, 1, 64, 64, state=False)
    d = cuda(x)
    leaves = [d[n].requires_grad_() for n in ("q", "k", "v", "dt", "A")]
    w, wn = randn(2, 64, 4, seed=1).cuda(), randn(64, seed=2).cuda()
    extra = torch.zeros(3, dtype=BF, device="cuda", requires_grad=True)
    up = randn(70 * 128 + 3, seed=3, dtype=BF).cuda()

    def outputs():
        o, _ = dn.ssm_scan(*leaves, d["dt_bias"], d["skip"])
        c, _ = dn.conv_silu_fn(leaves[2], w)
        return o, c, dn.gated_norm_fn(leaves[2], leaves[2], wn)

    for i in range(3):
        got = torch.autograd.grad(torch.cat([extra, outputs()[i].flatten()]), leaves, up, allow_unused=True)
        want = torch.autograd.grad(outputs()[i], leaves, up[3:].clone().view(1, 70, 2, 64), allow_unused=True)
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))
        assert got[2] is not None


def test_other_stream_and_graph_replays():
    """One training pass and one decoding step captured into graphs and replayed with eager work
    between the replays, inputs changed in place; every replay against the eager calls."""
    x, dO, dhT, _ = scan_inputs(1, 700, 2, 1, 64, 64, lens=[300, 0, 400])
    d, cu, dO, dhT = cuda(x), cu_of([300, 0, 400]), dO.cuda(), dhT.cuda()
    xc, w, b = randn(1, 700, 2, 64, seed=41, dtype=BF).cuda(), randn(2, 64, 4, seed=42).cuda(), randn(2, 64, seed=43).cuda()
    z, wn = randn(1, 700, 2, 64, seed=44, dtype=BF).cuda(), randn(64, seed=45).cuda()
    step_state, step_conv = randn(1, 2, 64, 64, seed=46).cuda(), randn(1, 3, 2, 64, seed=47, dtype=BF).cuda()

    def train():
        v, sT = dn.conv_silu(xc, w, b, None, cu)
        args = (d["q"], d["k"], v, d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"])
        o, hT = dn.ssm_fwd(*args, cu)
        y = dn.gated_norm(o, z, wn)
        do, dz, dwn = dn.gated_norm_bwd(o, z, wn, dO)
        g = dn.ssm_bwd(*args, do, dhT, cu)
        gc = dn.conv_silu_bwd(xc, w, b, None, g["dv"], None, cu)
        return [o, hT, y, dz, dwn, sT, *g.values(), *gc.values()]

    def step():
        v = dn.conv_silu_step(xc[:, 0], w, b, step_conv)
        return [dn.ssm_step(d["q"][:, 0], d["k"][:, 0], v, d["dt"][:, 0], d["A"], d["dt_bias"], d["skip"], step_state)]

    want = train()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = train()
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    start = (step_state.clone(), step_conv.clone())
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train()
    with torch.cuda.graph(graph2):
        out2 = step()
    for i in range(4):
        xc.copy_(randn(1, 700, 2, 64, seed=50 + i, dtype=BF))
        d["dt"].copy_(randn(1, 700, 2, seed=60 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, train()))
        for s, t in zip((step_state, step_conv), start):
            s.copy_(t)
        eager = step()
        after = (step_state.clone(), step_conv.clone())
        for s, t in zip((step_state, step_conv), start):
            s.copy_(t)
        graph2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2[0], eager[0])
        assert torch.equal(step_state, after[0]) and torch.equal(step_conv, after[1])


def test_scan_masked_steps_and_vanishing_decays():
    """Steps of minus infinity or the type's lowest value leave the state as it is, on the very
    first and last token too; decays past the float range clear it."""
    x, dO, dhT, ls = scan_inputs(1, 150, 2, 1, 64, 64)
    low = torch.finfo(F32).min
    for t, v in ((0, low), (1, -float("inf")), (63, low), (64, low), (65, -float("inf")), (100, -200.0), (149, low)):
        x["dt"][0, t] = v
    far = dict(x, dt=x["dt"].clamp_min(-1e5))  # softplus is 0 there in 64 bits as well
    val, bound = reference(far, ls, dO, dhT)
    d = cuda(x)
    args = (d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"])
    o, hT = dn.ssm_fwd(*args)
    gr = dn.ssm_bwd(*args, dO.cuda(), dhT.cuda())
    check(dict(gr, o=o, hT=hT), val, {k: b + 1e-37 for k, b in bound.items()}, list(val))
    state = d["h0"].clone()
    o1 = dn.ssm_step(d["q"][:, 1], d["k"][:, 1], d["v"][:, 1], d["dt"][:, 1], *args[4:7], state)
    assert torch.equal(state, d["h0"]) and torch.isfinite(o1).all()
    d["dt"].fill_(-float("inf"))
    o, hT = dn.ssm_fwd(*args)
    assert torch.equal(hT, d["h0"]) and torch.isfinite(o).all()
    d["dt"][0, 70, 1] = float("nan")
    _, hT = dn.ssm_fwd(*args)
    assert torch.isnan(hT[:, 1]).all() and torch.equal(hT[:, 0], d["h0"][:, 0])
    x, dO, dhT, ls = scan_inputs(1, 70, 2, 1, 64, 64, A=-3e38)
    val, bound = reference(x, ls, dO, dhT)
    d = cuda(x)
    args = (d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"])
    o, hT = dn.ssm_fwd(*args)
    gr = dn.ssm_bwd(*args, dO.cuda(), dhT.cuda())
    check(dict(gr, o=o, hT=hT), val, {k: b + 1e-37 for k, b in bound.items()}, list(val))


def test_step_sizes():
    # a first token with k = v = 1 leaves s in the state: within 6 half steps of fp32 (exponential 2,
    # its quotient and series 1.2 each, the sum with the step 1, rounded up) and without a bias
    dt = torch.cat([torch.linspace(-80, 30, 4000), torch.linspace(-8, 2, 4192)]).reshape(1024, 8).cuda()
    state = torch.zeros(1024, 8, 64, 64, device="cuda")
    one = torch.ones(1024, 8, 64, device="cuda")
    dn.ssm_step(one[:, :1].contiguous(), one[:, :1].contiguous(), one, dt, -torch.ones(8).cuda(), None, None, state)
    want = ref.softplus(dt.double())
    err = (state[:, :, 0, 0].double() - want) / want
    assert err.abs().max() <= 6 * ref.U32
    # the mean of n independent roundings is off by some 6 U32 / sqrt(n); four times that
    assert err.mean().abs() <= 4 * 6 * ref.U32 / 8192 ** 0.5
    assert torch.equal(state, state[:, :, :1, :1].expand_as(state))


def test_scan_of_a_pack_without_tokens():
    x, _, dhT, _ = scan_inputs(1, 0, 6, 2, 64, 128, lens=[0, 0, 0])
    d, cu = cuda(x), cu_of([0, 0, 0])
    o, hT = dn.ssm_fwd(**d, cu_seqlens=cu)
    assert o.numel() == 0 and torch.equal(hT, d["h0"])
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], d["v"], dhT.cuda(), cu)
    assert torch.equal(gr["dh0"].cpu(), dhT) and not gr["dA"].any() and not gr["dskip"].any()


@pytest.mark.parametrize("lens,tail", [([70, 0, 33], 97), ([2200, 5], 100), ([0, 0], 40)])
def test_rows_behind_the_last_sequence_stay(lens, tail):
    """Offsets that end before the rows do, called through the library itself, with NaN behind
    the last sequence and marked outputs."""
    H, G, dk, dv, n = 4, 1, 64, 64, sum(lens)
    x, dO, dhT, ls = scan_inputs(1, n, H, G, dk, dv, lens)
    val, bound = reference(x, ls, dO, dhT)
    pad = lambda t: torch.cat([t, torch.full((1, tail, *t.shape[2:]), float("nan"), dtype=t.dtype)], 1)  # noqa: E731
    d = {k: (pad(t) if k in ("q", "k", "v", "dt") else t).cuda() for k, t in x.items()}
    g, gT, cu = pad(dO).cuda(), dhT.cuda(), cu_of(lens)
    lib, T = dn.load_library(), n + tail
    s = ctypes.byref(dn._SsmShape(1, T, H, G, dk, dv, len(lens), 1))
    mark = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    out = dict(o=mark(d["v"]), hT=mark(d["h0"]))
    gr = dict(dq=mark(d["q"]), dk=mark(d["k"]), dv=mark(d["v"]), ddt=mark(d["dt"]), dA=mark(d["A"]),
              ddt_bias=mark(d["A"]), dskip=mark(d["A"]), dh0=mark(d["h0"]))
    ws = torch.empty(max(lib.dn_ssm_fwd_workspace(s), lib.dn_ssm_bwd_workspace(s)), dtype=torch.uint8, device="cuda")
    p = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    ins = p(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], cu)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.dn_ssm_fwd(s, *ins, *p(*out.values()), ws.data_ptr(), ws.numel(), st) == 0
    assert lib.dn_ssm_bwd(s, *ins, *p(g, gT, *gr.values()), ws.data_ptr(), ws.numel(), st) == 0
    for name, t in dict(gr, **out).items():
        if t.shape[:2] == (1, T):
            assert (t[:, n:] == 7).all(), name
    cut = {k: t[:, :n] if t.shape[:2] == (1, T) else t for k, t in dict(gr, **out).items()}
    check(cut, val, bound, list(val))
    xc, w, b = d["v"], randn(H, dv, 4, seed=2).cuda(), randn(H, dv, seed=3).cuda()
    y, sT, dx = mark(xc), xc.new_empty(len(lens), 3, H, dv), mark(xc)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    assert lib.dn_conv_silu(1, T, H, dv, 4, len(lens), 1, *p(xc, w, b), None, *p(cu, y, sT), st) == 0
    wsb = lib.dn_conv_silu_bwd_workspace(1, T, H, dv, 4)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    assert lib.dn_conv_silu_bwd(1, T, H, dv, 4, len(lens), 1, *p(xc, w, b), None, *p(cu, g), None, *p(dx, dw, db), None,
                                ws.data_ptr(), wsb, st) == 0
    assert (y[:, n:] == 7).all() and (dx[:, n:] == 7).all()
    y0, s0 = dn.conv_silu(xc[:, :n].contiguous(), w, b, None, cu)
    g0 = dn.conv_silu_bwd(xc[:, :n].contiguous(), w, b, None, g[:, :n].contiguous(), None, cu)
    assert torch.equal(y[:, :n], y0) and torch.equal(sT, s0) and torch.equal(dx[:, :n], g0["dx"])
    assert torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows against the same rows by themselves."""
    n, d = (1 << 31) // 4096 + 70, 4096
    x = torch.zeros(n, d, dtype=BF, device="cuda")
    end = randn(300, d, seed=1, dtype=BF).cuda()
    x[-300:] = end
    w = randn(d, seed=2).cuda()
    y = dn.gated_norm(x, x, w)
    assert torch.equal(y[-300:], dn.gated_norm(end, end, w)) and not y[:1000].any()
    dx, _, dw = dn.gated_norm_bwd(x, x, w, x)
    dx0, _, dw0 = dn.gated_norm_bwd(end, end, w, end)
    assert torch.equal(dx[-300:], dx0)
    # the same 300 terms |dy n g| <= r |x|^3, r < 1.2, added in two orders
    assert ((dw - dw0).abs() <= 2 * 300 * ref.U32 * 1.2 * (end.float().abs() ** 3).sum(0)).all()
    del y, dx
    wc, b = randn(32, 128, 4, seed=3).cuda(), randn(32, 128, seed=4).cuda()
    yc, sT = dn.conv_silu(x.view(1, n, 32, 128), wc, b)
    s0 = torch.zeros(1, 3, 32, 128, dtype=BF, device="cuda")
    y0, sT0 = dn.conv_silu(end.view(1, 300, 32, 128), wc, b, s0)
    assert torch.equal(yc[:, -300:], y0) and torch.equal(sT, sT0)
    gr = dn.conv_silu_bwd(x.view(1, n, 32, 128), wc, b, None, x.view(1, n, 32, 128))
    g0 = dn.conv_silu_bwd(end.view(1, 300, 32, 128), wc, b, s0, end.view(1, 300, 32, 128))
    assert torch.equal(gr["dx"][:, -300:], g0["dx"])
    del yc, gr
    # a long sequence and a short one behind it, whose results do not depend on the first
    sx, dO, dhT, _ = scan_inputs(1, 300, 32, 1, 64, 128, state=False, seed=5)
    val, bound = reference(sx, [300], dO)
    q = torch.zeros(1, n, 1, 64, dtype=BF, device="cuda")
    k, dt = torch.zeros_like(q), torch.zeros(1, n, 32, device="cuda")
    for t, name in ((q, "q"), (k, "k"), (dt, "dt")):
        t[:, -300:] = sx[name].cuda()
    x = x.view(1, n, 32, 128)
    x[:, -300:] = sx["v"].cuda()
    par = [sx[i].cuda() for i in ("A", "dt_bias", "skip")]
    cu = cu_of([n - 300, 300])
    o, hT = dn.ssm_fwd(q, k, x, dt, *par, None, cu)
    check(dict(o=o[:, -300:], hT=hT[1:]), val, bound, ["o", "hT"])
    assert not o[:, :1000].any() and not hT[0].any()
    o.zero_()
    o[:, -300:] = dO.cuda()
    gr = dn.ssm_bwd(q, k, x, dt, *par, None, o, None, cu)
    last = {i: g[:, -300:] if g.dim() > 1 else g for i, g in gr.items() if i != "dh0"}
    check(last, val, bound, list(last))


def test_two_streams_at_once():
    """Calls on two streams side by side, each with its own tensors and workspaces."""
    sets = [scan_inputs(1, 2500, 4, 2, 64, 64, seed=10 * i) for i in range(2)]
    sets = [(cuda(x), dO.cuda(), dhT.cuda()) for x, dO, dhT, _ in sets]

    def go(d, dO, dhT):
        args = (d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"])
        o, hT = dn.ssm_fwd(*args)
        return [o, hT, *dn.ssm_bwd(*args, dO, dhT).values()]

    want = [go(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(go(*s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_autograd_pass_in_a_graph_and_no_second_derivatives():
    x, dO, _, _ = scan_inputs(1, 130, 2, 1, 64, 64, state=False)
    d, dO = cuda(x), dO.cuda()
    w, wn = randn(2, 64, 4, seed=1).cuda(), randn(64, seed=2).cuda()
    leaves = [d["q"], d["k"], d["v"], d["dt"], d["A"], w, wn]

    def train():
        q, k, v, dt, A, w, wn = (t.detach().requires_grad_() for t in leaves)
        c, _ = dn.conv_silu_fn(v, w)
        o, _ = dn.ssm_scan(q, k, c, dt, A, d["dt_bias"], d["skip"])
        y = dn.gated_norm_fn(o, v, wn)
        return [y.detach(), *torch.autograd.grad(y, (q, k, v, dt, A, w, wn), dO)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train()
    for i in range(3):
        d["v"].copy_(randn(1, 130, 2, 64, seed=70 + i, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, train()))
    z = randn(2, 64, seed=3).cuda().requires_grad_()
    y = dn.gated_norm_fn(z, z, wn)
    (g,) = torch.autograd.grad(y.sum(), z, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_refusals_on_the_device():
    x, dO, _, _ = scan_inputs(1, 8, 4, 2, 64, 64)
    d = cuda(x)
    with pytest.raises(ValueError):
        dn.ssm_fwd(**dict(d, q=d["q"].transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(TypeError):
        dn.ssm_fwd(**dict(d, k=d["k"].float()))
    with pytest.raises(TypeError):
        dn.ssm_fwd(**dict(d, dt=d["dt"].double()))
    with pytest.raises(ValueError):
        dn.ssm_fwd(**dict(d, A=d["A"].cpu()))
    with pytest.raises(ValueError):
        dn.ssm_fwd(**dict(d, h0=d["h0"][..., :32].contiguous()))
    with pytest.raises(ValueError):  # three heads of queries do not divide four
        dn.ssm_fwd(**dict(d, q=torch.zeros(1, 8, 3, 64, dtype=BF).cuda()))
    with pytest.raises(TypeError):
        dn.ssm_fwd(**d, cu_seqlens=torch.tensor([0, 8]).cuda())
    with pytest.raises(dn.DnError):
        dn.ssm_fwd(**dict(d, q=torch.zeros(1, 8, 2, 32, dtype=BF).cuda(), k=torch.zeros(1, 8, 2, 32, dtype=BF).cuda(), h0=None))
    with pytest.raises(ValueError):
        dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], None, None, None, dO[..., :32].contiguous().cuda())
    xc = torch.zeros(1, 8, 2, 20).cuda()
    with pytest.raises(dn.DnError):
        dn.conv_silu(xc, torch.zeros(2, 20, 4).cuda())
    with pytest.raises(dn.DnError):
        dn.gated_norm(torch.zeros(2, 12).cuda(), torch.zeros(2, 12).cuda(), torch.ones(12).cuda())
    with pytest.raises(ValueError):
        dn.gated_norm(torch.zeros(2, 3, 16).cuda(), torch.zeros(2, 3, 16).cuda(), torch.ones(2, 16).cuda())
