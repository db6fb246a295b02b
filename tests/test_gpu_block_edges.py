"""The operators around the token mixers where calls meet: gates and parameters at the
ends of their ranges, outputs in place of inputs, calls side by side on two streams,
captured training passes, packs that end before their rows do, and refusals."""
import pytest
import torch

import block_ref as ref
import chunkwise_delta_rule_wy_amd as dn
from test_gpu_glr import BF, F32, both, check, cuda, inputs, reference

pytestmark = pytest.mark.gpu
E8 = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype,big", [(BF, 1e25), (F32, 3e38)])
def test_closed_gates_over_inputs_of_any_size(dtype, big):
    """Where a = 1 nothing of the token's input counts, in either direction."""
    d, dy, dhT, cu, _ = inputs(2, 200, 1, 16, dtype=dtype)
    d["r"][:, 60:100] = -torch.inf
    d["x"][:, 60:100] = 0
    want = both(d, dy, dhT, cu)
    d["x"][:, 60:100] = big
    got = both(d, dy, dhT, cu)
    for k in want:
        assert torch.isfinite(got[k]).all() and torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("power,lam", [(3e38, 5.0), (8.0, float("inf"))])
def test_largest_powers(power, lam):
    """An open gate forgets the state at once, a closed one keeps it all the same."""
    d, dy, dhT, cu, _ = inputs(1, 150, 1, 16, dtype=F32)
    d["lam"][:] = lam
    d["r"][:, 50:60] = -torch.inf
    got = both(d, dy, dhT, cu, power=power)
    want = torch.sigmoid(d["i"].double() + d["bi"].double()) * d["x"].double()
    want[:, 50:60] = want[:, 49:50]
    # an exponent of up to 12 rounded twice, and six roundings or approximations to a last digit or two
    assert ((got["y"].cpu().double() - want).abs() <= 32 * ref.U * want.abs()).all()
    for k in got:
        assert torch.isfinite(got[k]).all(), k
    assert not got["dr"].any() and not got["dlam"].any() and not got["dh0"].any()


def test_many_sequences():
    """More sequences than rows, most of them empty."""
    lens = ([1] + [0] * 3 + [2, 0]) * 700
    d, dy, dhT, cu, ls = inputs(1, sum(lens), 1, 8, lens)
    val, bound = reference(d, ls, dy, dhT)
    check(both(d, dy, dhT, cu), val, bound)


def test_step_of_the_most_sequences():
    B = 4 * 65535
    g = torch.Generator("cuda").manual_seed(3)
    x, r, i, h = (torch.randn(B, 1, 8, generator=g, device="cuda") for _ in range(4))
    lam = torch.zeros(1, 8, device="cuda")
    h1 = h.clone()
    y = dn.glr_step(x, r, i, lam, None, None, h1)
    h2 = h[-40:].clone()
    y2 = dn.glr_step(x[-40:].contiguous(), r[-40:].contiguous(), i[-40:].contiguous(), lam, None, None, h2)
    assert torch.equal(y[-40:], y2) and torch.equal(h1[-40:], h2) and torch.equal(y, h1)
    with pytest.raises(dn.DnError):
        dn.glr_step(*(torch.zeros(B + 1, 1, 8, device="cuda") for _ in range(3)), lam, None, None, torch.zeros(B + 1, 1, 8, device="cuda"))


def test_add_norm_in_place_of_its_inputs():
    lib, st = dn.load_library(), torch.cuda.current_stream().cuda_stream
    g = torch.Generator().manual_seed(5)
    seed = torch.tensor([3, 4]).cuda()
    for rows, D, E, R in ((700, 136, BF, BF), (700, 520, F32, F32), (2100, 4104, BF, BF), (33, 1032, BF, F32)):
        x, dy = (torch.randn(rows, D, generator=g).to(E).cuda() for _ in range(2))
        res, dh = (torch.randn(rows, D, generator=g).to(R).cuda() for _ in range(2))
        w = 1 + 0.1 * torch.randn(D, generator=g).cuda()
        y, h = dn.add_norm(x, res, w, p=0.25, seed=seed)
        dx, dres, dw = dn.add_norm_bwd(h, w, dy, dh, p=0.25, seed=seed)
        y8, scale, h8 = dn.norm8(x, res, w)
        e, r = dn._DTYPES[E], dn._DTYPES[R]
        a = lambda t: t.data_ptr()  # noqa: E731
        x2, res2, dy2, dh2, res3 = x.clone(), res.clone(), dy.clone(), dh.clone(), res.clone()
        z8, s8, dw2 = torch.empty_like(y8), torch.empty_like(scale), torch.empty_like(dw)
        ws = torch.empty(lib.dn_add_norm_bwd_workspace(rows, D), dtype=torch.uint8, device="cuda")
        assert lib.dn_add_norm(rows, D, e, r, a(x2), a(res2), a(w), 1e-5, 0.25, a(seed), a(x2), a(res2), st) == 0
        assert lib.dn_add_norm_bwd(rows, D, e, r, a(h), a(w), 1e-5, 0.25, a(seed), a(dy2), a(dh2), a(dy2), a(dh2), a(dw2), a(ws),
                                   ws.numel(), st) == 0
        assert lib.dn_norm8(rows, D, e, r, a(x), a(res3), a(w), 1e-5, a(z8), a(s8), a(res3), st) == 0
        torch.cuda.synchronize()
        for got, want in ((x2, y), (res2, h), (dy2, dx), (dh2, dres), (dw2, dw), (z8.float(), y8.float()), (s8, scale), (res3, h8)):
            assert torch.equal(got, want), (rows, D)


@pytest.mark.parametrize("M,N", [(5, 40), (60, 67), (100, 1000), (300, 1001), (1030, 4088), (4090, 4000), (3999, 4091)])
def test_product_in_place_of_its_residual(M, N):
    g = torch.Generator().manual_seed(6)
    x, w = (torch.randint(-2, 3, (n, 144), generator=g).float().to(E8).cuda() for n in (M, N))
    xs, ws = torch.full((M,), 0.25, device="cuda"), torch.ones(N, device="cuda")
    r = torch.randn(M, N, generator=g).to(BF).cuda()
    want = dn.linear8(x, xs, w, ws, residual=r)
    a = lambda t: t.data_ptr()  # noqa: E731
    assert dn.load_library().dn_linear8(M, N, 144, a(x), a(xs), a(w), a(ws), None, a(r), 0, a(r), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(r, want)


def test_calls_side_by_side():
    """Two streams with calls of their own at the same time: no memory is shared between calls."""
    sets = []
    for n in range(2):
        d, dy, dhT, cu, _ = inputs(1, 6000, 1, 64, [2500, 0, 3400], seed=n)
        c = cuda(d)
        g = torch.Generator().manual_seed(20 + n)
        x, res, ey = (torch.randn(3000, 512, generator=g).to(BF).cuda() for _ in range(3))
        w = torch.ones(512).cuda()
        w8, ws = dn.norm8(torch.randn(1024, 512, generator=g).cuda())[:2]
        sets.append((c, dy.cuda(), dhT.cuda(), cu.cuda(), x, res, ey, w, w8, ws))

    def work(c, dy, dhT, cu, x, res, ey, w, w8, ws):
        y, hT = dn.glr_fwd(**c, cu_seqlens=cu)
        gr = dn.glr_bwd(*c.values(), dy, dhT, cu)
        y8, s, h = dn.norm8(x, res, w)
        return [y, hT, *gr.values(), *dn.add_norm_bwd(h, w, ey), dn.linear8(y8, s, w8, ws, act="silu")]

    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                got[n].append(work(*sets[n]))
    torch.cuda.synchronize()
    for n in range(2):
        for out in got[n]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[n])), n


def test_captured_training_pass():
    """A layer's pass through autograd, captured with fresh leaves and replayed with other values and seeds."""
    g = torch.Generator().manual_seed(7)
    B, T, H, D, W = 1, 300, 2, 32, 64
    x, res, r, i, dy = (torch.randn(B, T, W, generator=g).to(BF).cuda() for _ in range(5))
    w, lam = 1 + 0.1 * torch.randn(W, generator=g).cuda(), torch.randn(H, D, generator=g).cuda() - 4
    cu, seed = torch.tensor([0, 100, 250], dtype=torch.int32).cuda(), torch.tensor([5, 6]).cuda()

    def step():
        leaf = [t.detach().clone().requires_grad_() for t in (x, res, w, r, i, lam)]
        y, h = dn.add_norm_fn(leaf[0], leaf[1], leaf[2], p=0.1, seed=seed)
        heads = lambda t: t.reshape(B, T, H, D)  # noqa: E731
        o, hT = dn.glr_scan(heads(y), heads(leaf[3]), heads(leaf[4]), leaf[5], cu_seqlens=cu)
        out, _ = dn.add_norm_fn(o.reshape(B, T, W), h, leaf[2], p=0.1, seed=seed)
        return [out.detach(), hT.detach(), *torch.autograd.grad(out, leaf, dy)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        seed += 1
        x.mul_(-1.25)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.isfinite(a).all() and torch.equal(a, b), k


def test_padded_batch_through_autograd():
    """A pack that ends before its rows do: the rows behind it take no part, whatever they hold."""
    d, dy, dhT, cu, ls = inputs(1, 400, 1, 24, [100, 0, 150])
    val, bound = reference(d, ls, dy, dhT)
    for k in ("x", "r", "i"):
        d[k][0, 250:] = torch.nan
    c = {k: v.cuda().requires_grad_() for k, v in d.items()}
    y, hT = dn.glr_scan(*c.values(), cu.cuda())
    dy[0, 250:] = torch.nan
    grads = torch.autograd.grad([y, hT], list(c.values()), [dy.cuda(), dhT.cuda()])
    check(dict(zip(("dx", "dr", "di", "dlam", "dbr", "dbi", "dh0"), grads), y=y.detach(), hT=hT.detach()), val, bound)
    for t in (y,) + grads[:3]:
        assert not t[0, 250:].any()


def test_rows_without_a_finite_norm_in_eight_bits():
    """NaN stays in its place where the row is not normed; an infinity's row has an infinite scale."""
    x = torch.ones(4, 64, device="cuda")
    x[1, 5], x[2, 9] = torch.nan, torch.inf
    y, s, _ = dn.norm8(x)
    assert torch.isnan(y[1, 5].float()) and (y[1, :5].float() == 448).all() and s[1] == s[0] == 1 / 448
    assert torch.isinf(s[2]) and torch.isnan(y[2, 9].float()) and (y[3].float() == 448).all()


def test_refusals():
    z = lambda *s, t=F32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    x, p, st = z(2, 6, 2, 8, t=BF), z(2, 8), z(2, 2, 8)
    cu = torch.tensor([0, 6], dtype=torch.int32)
    E, V = TypeError, ValueError
    bad = [
        (E, lambda: dn.glr_fwd(x, x.float(), x, p)), (E, lambda: dn.glr_fwd(x, x, x, p.to(BF))),
        (V, lambda: dn.glr_fwd(x, x[:, :5], x, p)), (V, lambda: dn.glr_fwd(x, x, x.transpose(1, 2), p)),
        (V, lambda: dn.glr_fwd(x.transpose(2, 3), x, x, p)), (V, lambda: dn.glr_fwd(x, x, x, p.cpu())),
        (V, lambda: dn.glr_fwd(x, x, x, z(8, 2))), (V, lambda: dn.glr_fwd(x, x, x, p, z(8))),
        (V, lambda: dn.glr_fwd(x, x, x, p, h0=st[:1])), (V, lambda: dn.glr_fwd(x, x, x, p, h0=st[:1].expand(2, 2, 8))),
        (V, lambda: dn.glr_fwd(x, x, x, p, cu_seqlens=cu.cuda())), (V, lambda: dn.glr_fwd(x[:1], x[:1], x[:1], p, cu_seqlens=cu)),
        (E, lambda: dn.glr_fwd(x[:1], x[:1], x[:1], p, cu_seqlens=cu.long().cuda())),
        (V, lambda: dn.glr_fwd(x[:1], x[:1], x[:1], p, cu_seqlens=[0, 6])),
        (V, lambda: dn.glr_fwd(x, x, x, p, states=z(2, 2, 8))), (E, lambda: dn.glr_fwd(x, None, x, p)),
        (E, lambda: dn.glr_bwd(x, x, x, p, None, None, None, None)), (V, lambda: dn.glr_bwd(x, x, x, p, None, None, None, x[:1])),
        (E, lambda: dn.glr_bwd(x, x, x, p, None, None, None, x, dhT=st.to(BF))),
        (V, lambda: dn.glr_step(x[:, 0], x[:, 0], x[:, 0], p, None, None, st)),  # slices of a token: not contiguous
        (E, lambda: dn.glr_step(x[0], x[0], x[0], p, None, None, None)),
        (V, lambda: dn.glr_step(x[0], x[0], x[0], p, None, None, st)),
        (V, lambda: dn.add_norm(x, x[:1], z(8))), (V, lambda: dn.add_norm(x, x, p)), (E, lambda: dn.add_norm(x, x, None)),
        (E, lambda: dn.add_norm(x.float(), x, z(8))), (E, lambda: dn.add_norm(x, x, z(8, t=BF))),
        (V, lambda: dn.add_norm(z(4, 0), None, z(0))), (V, lambda: dn.add_norm(z(4, 16)[:, ::2], None, z(8))),
        (V, lambda: dn.add_norm(x, x, z(8), p=1.0)), (V, lambda: dn.add_norm(x, x, z(8), p=float("nan"))),
        (E, lambda: dn.add_norm(x, x, z(8), p=0.5)), (V, lambda: dn.add_norm(x, x, z(8), p=0.5, seed=torch.tensor([1, 2]))),
        (E, lambda: dn.add_norm(x, x, z(8), p=0.5, seed=z(2))), (V, lambda: dn.add_norm(x, x, z(8), p=0.5, seed=z(3, t=torch.int64))),
        (V, lambda: dn.add_norm_bwd(x, z(8), x, dh=x[:1])), (E, lambda: dn.add_norm_bwd(x, z(8), x, dh=x.float())),
        (E, lambda: dn.add_norm_bwd(None, z(8), x)), (E, lambda: dn.norm8(x.half())), (V, lambda: dn.norm8(x, x.cpu())),
        (V, lambda: dn.norm8(z(3, 0))),
    ]
    w8, x8 = z(24, 32).to(E8), z(3, 32).to(E8)
    a = dict(x=x8, xs=z(3), w=w8, ws=z(24))
    for err, kw in ((V, dict(xs=z(4))), (E, dict(xs=z(3, t=BF))), (V, dict(ws=z(3))), (V, dict(w=z(24, 16).to(E8))), (E, dict(w=z(24, 32))),
                    (V, dict(w=z(32, 24).to(E8).t())), (V, dict(bias=z(3))), (E, dict(residual=z(3, 24))), (V, dict(residual=z(24, 3, t=BF).t())),
                    (V, dict(act="tanh")), (V, dict(act=None)), (E, dict(xs=None)), (V, dict(xs=z(3).cpu()))):
        bad.append((err, lambda kw=kw: dn.linear8(**{**a, **kw})))
    for n, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            print("accepted: number", n)
    # sizes and addresses that the library refuses
    odd = z(1, 1, 1, 17, t=BF)[..., 1:9].contiguous().new_zeros(4 * 8 + 1)[1:33].view(1, 4, 1, 8)
    for call in (lambda: dn.glr_fwd(odd, odd, odd, p[:1]), lambda: dn.glr_fwd(*[z(1, 4, 1, 12)] * 3, z(1, 12)),
                 lambda: dn.glr_fwd(x, x, x, p, power=0.0), lambda: dn.add_norm(z(2, 8200), None, z(8200)),
                 lambda: dn.add_norm(odd, None, z(8)), lambda: dn.add_norm(x, x, z(8), p=1 - 1e-9, seed=z(2, t=torch.int64)),
                 lambda: dn.linear8(z(3, 24).to(E8), z(3), z(8, 24).to(E8), z(8))):
        with pytest.raises(dn.DnError):
            call()


@pytest.mark.parametrize("B,T,H,lens", [(2, 1024, 104, None), (1, 1500, 104, None), (1, 1500, 128, [700, 0, 790])])
def test_directions_cut_in_different_ways(B, T, H, lens):
    """Where the backward pass cuts sequences that the forward pass walks through, with and without kept states."""
    d, dy, dhT, cu, ls = inputs(B, T, H, 64 if B == 1 else 32, lens)
    got, again = both(d, dy, dhT, cu), both(d, dy, dhT, cu, keep=False)
    for k in got:
        assert torch.equal(got[k], again[k]), k
    C = d["lam"].numel()
    pick = [0, 63, 64, C - 1]
    col = lambda v: v.reshape(*v.shape[:-2], -1)[..., pick][..., None, :]  # noqa: E731
    val, bound = reference({k: v if v is None else col(v) for k, v in d.items()}, ls, col(dy), col(dhT))
    check({k: col(v).cpu() for k, v in got.items()}, val, bound)
