"""GPU parity of the residual's addition with dropout and norm, and of its 8-bit
form, with the 64-bit reference, and the ways a program uses them."""
import pytest
import torch

import block_ref as ref
import chunkwise_delta_rule_wy_amd as dn

pytestmark = pytest.mark.gpu
BF, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SEED = [0x0123456789ABCDEF, -5]


def inputs(rows, D, E, R, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res, dy, dh = n(rows, D).to(E), n(rows, D).to(R), n(rows, D).to(E), n(rows, D).to(R)
    return x, res, 1 + 0.2 * n(D), dy, dh


def within(got, val, bound, name):
    assert torch.isfinite(got).all(), name
    w = ref.worst(got, val, bound)
    assert w <= 1, (name, w)


TYPES = [(BF, BF), (BF, F32), (F32, F32)]
WIDTHS = [8, 24, 64, 72, 136, 256, 264, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192]


@pytest.mark.parametrize("E,R", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_sum_norm_and_gradients(D, E, R):
    rows, eps = (37, 1e-5) if D < 4000 else (5, 1e-3)
    x, res, w, dy, dh = inputs(rows, D, E, R, D)
    y, h = dn.add_norm(x.cuda(), res.cuda(), w.cuda(), eps)
    assert y.dtype == E and h.dtype == R
    # the sum: one rounding of each type's
    total = x.double() + res.double()
    within(h, total, ref.half(R) * total.abs() + 2 * ref.U * (x.double().abs() + res.double().abs()), "h")
    hd, wd, dyd, dhd = h.cpu().double(), w.double(), dy.double(), dh.double()
    want, dres, dw = ref.norm(hd, wd, eps, dyd, dhd)
    bound = ref.norm_bounds(hd, wd, eps, E, R, dyd, dhd, torch.ones(1, dtype=torch.float64))
    within(y, want, bound["y"], "y")
    gx, gr, gw = dn.add_norm_bwd(h, w.cuda(), dy.cuda(), dh.cuda(), eps)
    assert gx.dtype == E and gr.dtype == R and (gx is gr) == (E is R)
    within(gr, dres, bound["dres"], "dres")
    within(gx, dres, bound["dx"], "dx")
    within(gw, dw, bound["dw"], "dw")


@pytest.mark.parametrize("E,R", TYPES)
@pytest.mark.parametrize("rows,D,p", [(33, 72, 0.1), (5, 1024, 0.5), (3, 4104, 0.25), (9, 64, 1e-6), (9, 128, 0.999)])
def test_dropout(rows, D, p, E, R):
    x, res, w, dy, dh = inputs(rows, D, E, R, 3)
    seed = torch.tensor(SEED).cuda()
    keep = ref.keep_factors(SEED, p, rows, D)
    y, h = dn.add_norm(x.cuda(), res.cuda(), w.cuda(), p=p, seed=seed)
    total = res.double() + keep * x.double()
    within(h, total, ref.half(R) * total.abs() + 3 * ref.U * (keep * x.double().abs() + res.double().abs()), "h")
    hd, wd, dyd, dhd = h.cpu().double(), w.double(), dy.double(), dh.double()
    want, dres, dw = ref.norm(hd, wd, 1e-5, dyd, dhd)
    bound = ref.norm_bounds(hd, wd, 1e-5, E, R, dyd, dhd, keep)
    within(y, want, bound["y"], "y")
    gx, gr, gw = dn.add_norm_bwd(h, w.cuda(), dy.cuda(), dh.cuda(), p=p, seed=seed)
    within(gr, dres, bound["dres"], "dres")
    within(gx, keep * dres, bound["dx"], "dx")
    within(gw, dw, bound["dw"], "dw")


def test_mask_follows_seed_stream_and_place():
    ones = torch.ones(400, 264, device="cuda")
    w = torch.ones(264, device="cuda")
    mask = lambda s, x=ones: dn.add_norm(x, None, w, p=0.3, seed=torch.tensor(s).cuda())[1]  # noqa: E731
    a = mask(SEED)
    assert torch.equal(a, mask(SEED)) and torch.equal(a[:7], mask(SEED, ones[:7]))
    others = [mask([SEED[0] + 1, SEED[1]]), mask([SEED[0], SEED[1] + 1]), mask([SEED[0] ^ (1 << 40), SEED[1]]), mask([SEED[0], SEED[1] ^ (1 << 50)])]
    # independent draws of 0.3 agree in 0.58 of the places; 105600 of them give a deviation of 0.0015
    for o in others:
        assert abs((o == a).double().mean().item() - 0.58) < 6 * 0.0016
    assert abs((a == 0).double().mean().item() - 0.3) < 6 * 0.0015
    # and no row or column stands out: 6 deviations of its mean
    assert ((a == 0).double().mean(0) - 0.3).abs().max() < 6 * (0.21 / 400) ** 0.5
    assert ((a == 0).double().mean(1) - 0.3).abs().max() < 6 * (0.21 / 264) ** 0.5
    assert torch.equal(mask(SEED, ones.to(BF)).float() > 0, a > 0)  # whatever the type


def test_mask_of_far_rows():
    # blocks past 32 bits of the counter: the last rows of 2^35 values in pieces cannot be held, so that the
    # counter's upper word is tested at the widest row count that fits
    rows, D = 1 << 21, 4096
    x = torch.ones(rows, D, dtype=BF, device="cuda")
    seed = torch.tensor(SEED).cuda()
    h = dn.add_norm(x, None, torch.ones(D, device="cuda"), p=0.5, seed=seed)[1]
    keep = ref.keep_factors(SEED, 0.5, 2, D, rows - 2)
    assert torch.equal(h[-2:].cpu().double(), keep)


def test_without_residual():
    x, _, w, dy, dh = inputs(11, 72, BF, BF)
    y, h = dn.add_norm(x.cuda(), None, w.cuda())
    assert torch.equal(h.cpu(), x)
    y2, _ = dn.add_norm(x.cuda(), torch.zeros_like(x).cuda(), w.cuda())
    assert torch.equal(y, y2)
    y8, s8, h8 = dn.norm8(x.cuda(), None, w.cuda())
    z8, t8, _ = dn.norm8(x.cuda(), torch.zeros_like(x).cuda(), w.cuda())
    assert torch.equal(y8.float(), z8.float()) and torch.equal(s8, t8) and torch.equal(h8.cpu(), x)


def test_empty_and_zero_rows():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    y, h = dn.add_norm(e, e, w)
    assert y.shape == h.shape == (0, 64)
    _, _, dw = dn.add_norm_bwd(e, w, e)
    assert not dw.any()
    y8, s, _ = dn.norm8(e, None, w)
    assert y8.shape == (0, 64) and s.shape == (0,)
    z = torch.zeros(3, 64, device="cuda")
    y, _ = dn.add_norm(z, z, w)
    assert not y.any()
    dx, _, _ = dn.add_norm_bwd(z, w, torch.ones_like(z))
    assert torch.isfinite(dx).all()
    y8, s, _ = dn.norm8(z, z, w)
    assert not y8.float().any() and (s > 0).all() and torch.isfinite(1 / s).all()


def test_leading_sizes_and_nan_rows():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 5, 40, generator=g).to(BF).cuda()
    w = torch.ones(40, device="cuda")
    y, h = dn.add_norm(x, x, w)
    y8, s, _ = dn.norm8(x, x, w)
    assert y.shape == h.shape == y8.shape == x.shape and s.shape == (2, 3, 5)
    bad = x.clone()
    bad[1, 2, 3, 4] = torch.nan
    y2, _ = dn.add_norm(bad, x, w)
    z8, t, _ = dn.norm8(bad, x, w)
    assert torch.isnan(y2[1, 2, 3]).all() and torch.isnan(z8[1, 2, 3].float()).all()
    keep = torch.ones(2, 3, 5, dtype=torch.bool)
    keep[1, 2, 3] = False
    assert torch.equal(y2[keep.cuda()], y[keep.cuda()]) and torch.equal(t[keep.cuda()], s[keep.cuda()])


def steps(y8):
    """The step of 8-bit floats at these values: 2^-3 of the power of two, 2^-9 at the least."""
    return torch.exp2(torch.floor(torch.log2(y8.abs().clamp(min=2.0 ** -6))) - 3)


@pytest.mark.parametrize("E,R", TYPES)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D", WIDTHS)
def test_rows_in_eight_bits(D, norm, E, R):
    rows = 37 if D < 4000 else 5
    x, res, w, _, _ = inputs(rows, D, E, R, D + 1)
    x[1] *= 1e-3
    w = w if norm else None
    y8, scale, h = dn.norm8(x.cuda(), res.cuda(), None if w is None else w.cuda())
    assert y8.dtype == E8 and h.dtype == R
    _, h2 = dn.add_norm(x.cuda(), res.cuda(), torch.ones(D).cuda())
    assert torch.equal(h, h2)
    y = ref.norm(h.cpu().double(), None if w is None else w.double(), 1e-5)
    top = y.abs().amax(-1) / 448
    assert ((scale.cpu().double() - top).abs() <= 40 * ref.U * top).all()
    # half a step around the exact quotient, and its own error before the rounding
    q = y / scale.cpu().double()[:, None]
    got = y8.cpu().double()
    assert ((got - q).abs() <= steps(q) / 2 * (1 + 1e-5) + 44 * ref.U * q.abs()).all()
    assert (got.abs().amax(-1) == 448).all()


def test_eight_bits_of_all_values():
    # every finite 8-bit value comes back, and the halves between neighbours go to the even one
    codes = torch.arange(256, dtype=torch.uint8).view(E8).float()
    vals = codes[torch.isfinite(codes)].unique()
    mid = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mid, torch.tensor([448.0] * 3)])
    x = torch.cat([x, torch.zeros(-len(x) % 8)])[None]
    y8, scale, _ = dn.norm8(x.cuda())
    assert scale.item() == 1
    assert torch.equal(y8.cpu().float(), x.to(E8).float())


def test_autograd():
    x, res, w, dy, dh = inputs(20, 136, F32, F32, 9)
    seed = torch.tensor(SEED).cuda()
    for p, residual in ((0.0, True), (0.2, True), (0.2, False), (0.0, False)):
        leaves = [x.cuda().requires_grad_()] + ([res.cuda().requires_grad_()] if residual else []) + [w.cuda().requires_grad_()]
        y, h = dn.add_norm_fn(leaves[0], leaves[1] if residual else None, leaves[-1], p=p, seed=seed)
        got = torch.autograd.grad([y, h], leaves, [dy.cuda(), dh.cuda()])
        keep = ref.keep_factors(SEED, p, 20, 136)
        hd = h.detach().cpu().double()
        _, dres, dw = ref.norm(hd, w.double(), 1e-5, dy.double(), dh.double())
        b = ref.norm_bounds(hd, w.double(), 1e-5, F32, F32, dy.double(), dh.double(), keep)
        within(got[0], keep * dres, b["dx"], "dx")
        within(got[-1], dw, b["dw"], "dw")
        if residual:
            within(got[1], dres, b["dres"], "dres")
    # only one of the outputs used
    a = x.cuda().requires_grad_()
    y, h = dn.add_norm_fn(a, res.cuda(), w.cuda(), p=0.2, seed=seed)
    (g,) = torch.autograd.grad(h.sum(), [a])
    assert torch.equal(g.cpu().double(), ref.keep_factors(SEED, 0.2, 20, 136).float().double())
    # a seed that changed in between is noticed
    y, h = dn.add_norm_fn(a, res.cuda(), w.cuda(), p=0.2, seed=seed)
    seed += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_graph_replays_follow_the_seed():
    x, res, w, dy, dh = (t.cuda() for t in inputs(300, 520, BF, F32, 4))
    seed = torch.tensor(SEED).cuda()

    def step():
        y, h = dn.add_norm(x, res, w, p=0.1, seed=seed)
        return (y, h) + dn.add_norm_bwd(h, w, dy, dh, p=0.1, seed=seed) + dn.norm8(x, res, w)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        seed += 1
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.float(), b.float())


@pytest.mark.parametrize("E", [BF, F32])
@pytest.mark.parametrize("rows,D", [(4000, 64), (300, 520), (700, 1000), (200, 1032), (500, 4096), (60, 8192)])
def test_eight_bits_are_the_rounded_quotient(rows, D, E):
    """Without norm y8 is the fp32 quotient h / scale rounded to nearest even, bit for bit: scales that are no powers of
    two put many quotients of bf16 values next to, and onto, the halves between 8-bit values."""
    x, res, _, _, _ = inputs(rows, D, E, E, 77)
    x[::7] *= 1e-30  # a row's values around the least scale, and below the fp32 range
    x[1::7] *= 1e36
    x[2::7] *= 1e-36
    res[::7], res[1::7], res[2::7] = 0, 0, 0
    for r in (None, res):
        y8, scale, h = dn.norm8(x.cuda(), None if r is None else r.cuda())
        h, scale = h.cpu().float(), scale.cpu()
        assert torch.equal(scale, h.abs().amax(-1).clamp(min=1e-30) / 448)
        want = (h / scale[:, None]).to(E8).float()
        got = y8.cpu().float()
        assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("E,R", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256, 520, 1032, 2048, 4096, 8192])
def test_normed_rows_with_an_infinity_in_eight_bits(D, E, R):
    """An infinite scale, and NaN as a whole; the other rows as without it."""
    x, res, w, _, _ = inputs(9, D, E, R, D)
    clean = dn.norm8(x.cuda(), res.cuda(), w.cuda())
    x[2, D - 1], res[5, D // 2], x[7, 0] = torch.inf, -torch.inf, -torch.inf
    y8, scale, h = dn.norm8(x.cuda(), res.cuda(), w.cuda())
    bad = [2, 5, 7]
    assert (scale[bad] == torch.inf).all() and torch.isnan(y8[bad].float()).all()
    keep = [0, 1, 3, 4, 6, 8]
    assert torch.equal(y8[keep].float(), clean[0][keep].float()) and torch.equal(scale[keep], clean[1][keep])
    assert torch.equal(h[keep], clean[2][keep]) and torch.isinf(h[[2, 5, 7], [D - 1, D // 2, 0]]).all()


def test_mask_past_32_bits_of_blocks():
    """2^32 blocks of eight values and some, whose numbers reach into the counter's upper word (2^21 rows of 4096 values
    end at 2^30 of them).  64 GiB, dropped and normed in place."""
    lib, rows, D, n = dn.load_library(), (1 << 22) + 3, 8192, 5
    x = torch.ones(rows, D, dtype=BF, device="cuda")
    seed, w = torch.tensor(SEED).cuda(), torch.ones(D, device="cuda")
    a = lambda t: t.data_ptr()  # noqa: E731
    assert lib.dn_add_norm(rows, D, 1, 1, a(x), None, a(w), 1e-5, 0.5, a(seed), a(x), None, torch.cuda.current_stream().cuda_stream) == 0
    last, first = x[-n:].float().cpu(), x[:n].float().cpu()
    del x
    torch.cuda.empty_cache()
    assert torch.equal(last > 0, ref.keep_factors(SEED, 0.5, n, D, rows - n) > 0)
    assert torch.equal(first > 0, ref.keep_factors(SEED, 0.5, n, D) > 0)
    # rows 0, 1, 2 and the last three have the same lower words
    assert not torch.equal(last[-3:] > 0, first[:3] > 0)


@pytest.mark.parametrize("E,R", TYPES)
def test_dropped_values_that_are_not_finite(E, R):
    """A dropped value is multiplied by 0, which gives NaN for one that is not finite, forwards and backwards."""
    x, res, w, dy, dh = inputs(6, 128, E, R, 1)
    keep = ref.keep_factors(SEED, 0.5, 6, 128)
    seed = torch.tensor(SEED).cuda()
    r = 3
    drop, kept = (int((keep[r] == v).nonzero()[0]) for v in (0.0, 2.0))
    x[r, drop] = x[r, kept] = torch.inf
    h = dn.add_norm(x.cuda(), res.cuda(), w.cuda(), p=0.5, seed=seed)[1]
    assert torch.isnan(h[r, drop]) and h[r, kept] == torch.inf
    other = [0, 1, 2, 4, 5]
    assert torch.isfinite(h[other]).all()
    dh[r, drop] = dh[r, kept] = torch.inf
    dx, dres, _ = dn.add_norm_bwd(res.cuda(), w.cuda(), dy.cuda(), dh.cuda(), p=0.5, seed=seed)
    assert torch.isnan(dx[r, drop]) and dx[r, kept] == torch.inf and (dres[r, [drop, kept]] == torch.inf).all()
    assert torch.isfinite(dx[other]).all()


@pytest.mark.parametrize("E,R", TYPES)
def test_rows_whose_squares_pass_the_range(E, R):
    x, res, w, _, _ = inputs(4, 128, E, R, 2)
    x[1], res[1] = 1e25, 0
    y, h = dn.add_norm(x.cuda(), res.cuda(), w.cuda())
    y8, scale, _ = dn.norm8(x.cuda(), res.cuda(), w.cuda())
    assert not y[1].any() and not y8[1].float().any() and scale[1] == torch.tensor(1e-30) / 448
    assert torch.isfinite(h).all() and (scale[[0, 2, 3]] > 1e-4).all() and y[[0, 2, 3]].any(1).all()
