"""GPU parity of the gated linear recurrence with the 64-bit reference, within
the bounds that its roundings allow, and the ways a program uses it."""
import pytest
import torch

import block_ref as ref
import chunkwise_delta_rule_wy_amd as dn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, H, D, lens=None, state=True, dtype=BF, seed=0, bias=True, gate=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N = len(lens) if lens is not None else B
    d = dict(x=n(B, T, H, D).to(dtype), r=(gate * n(B, T, H, D)).to(dtype), i=n(B, T, H, D).to(dtype))
    keep = 0.9 + 0.0999 * torch.rand(H, D, generator=g)
    d["lam"] = torch.log(torch.expm1(-torch.log(keep) / 8))
    d["br"], d["bi"] = (n(H, D), n(H, D)) if bias else (None, None)
    d["h0"] = n(N, H, D) if state else None
    dy, dhT = n(B, T, H, D).to(dtype), n(N, H, D) if state else None
    cu = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    return d, dy, dhT, cu, lens if lens is not None else [T] * B


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def reference(d, lens, dy=None, dhT=None, power=8.0):
    C = d["lam"].numel()
    f = lambda t, n: None if t is None else t.double().reshape(n, C)  # noqa: E731
    rows = d["x"].numel() // C
    v = lambda t: None if t is None else t.double().reshape(C)  # noqa: E731
    return ref.glr(f(d["x"], rows), f(d["r"], rows), f(d["i"], rows), v(d["lam"]), v(d["br"]), v(d["bi"]),
                   f(d["h0"], len(lens)), lens, power, f(dy, rows), f(dhT, len(lens)), d["x"].dtype)


def check(got, val, bound, names=None):
    for k in names or val:
        g = got[k]
        assert torch.isfinite(g).all(), k
        w = ref.worst(g.reshape(val[k].shape), val[k], bound[k])
        assert w <= 1, (k, w)


def both(d, dy, dhT, cu, power=8.0, keep=True):
    c, dy = cuda(d), dy.cuda()
    dhT, cu = None if dhT is None else dhT.cuda(), None if cu is None else cu.cuda()
    states = dn.glr_states(c["x"]) if keep else None
    y, hT = dn.glr_fwd(**c, cu_seqlens=cu, power=power, states=states)
    gr = dn.glr_bwd(*c.values(), dy, dhT, cu, power=power, states=states)
    torch.cuda.synchronize()
    return dict(gr, y=y, hT=hT)


SHAPES = [
    # B, T, H, D, packed lengths, carried state
    (1, 1, 1, 8, None, True),
    (3, 1, 2, 8, None, False),
    (2, 7, 1, 40, None, True),
    (2, 127, 1, 72, None, True),
    (1, 128, 1, 64, None, False),
    (1, 129, 3, 24, None, True),
    (5, 200, 1, 136, None, True),     # short sequences share segments
    (2, 513, 1, 64, None, True),      # cut by themselves, a ragged last tile
    (2, 1100, 2, 40, None, False),
    (1, 300, 2, 40, [0, 1, 63, 64, 0, 65, 107, 0], True),
    (1, 700, 1, 64, [1, 1, 600, 98], False),
    (1, 5, 1, 8, [0, 0, 5], True),
    (1, 260, 1, 16, [1] * 130 + [0, 0] + [2] * 65, True),
    (1, 900, 1, 24, [128, 128, 256, 384, 4], True),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,D,lens,state", SHAPES)
def test_recurrence_and_gradients(B, T, H, D, lens, state, dtype):
    d, dy, dhT, cu, ls = inputs(B, T, H, D, lens, state, dtype)
    val, bound = reference(d, ls, dy, dhT)
    got = both(d, dy, dhT, cu)
    assert got["y"].dtype == got["dx"].dtype == got["dr"].dtype == got["di"].dtype == dtype
    check(got, val, bound)


@pytest.mark.parametrize("B,T,lens", [(2, 600, None), (7, 33, None), (1, 400, [100, 0, 300])])
def test_recomputed_states_give_the_same_gradients(B, T, lens):
    d, dy, dhT, cu, _ = inputs(B, T, 1, 72, lens)
    a, b = both(d, dy, dhT, cu), both(d, dy, dhT, cu, keep=False)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_without_biases_and_states():
    d, dy, _, _, ls = inputs(2, 90, 2, 16, state=False, bias=False)
    val, bound = reference(d, ls, dy)
    got = both(d, dy, None, None)
    assert got["dbr"] is None and got["dbi"] is None
    check(got, val, bound, ["y", "hT", "dx", "dr", "di", "dlam", "dh0"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("power,gate", [(8.0, 6.0), (0.01, 1.0), (1e-4, 1.0), (300.0, 3.0), (1e4, 1.0)])
def test_decays_from_none_to_at_once(power, gate, dtype):
    d, dy, dhT, cu, ls = inputs(1, 400, 1, 24, [250, 150], dtype=dtype, gate=gate)
    val, bound = reference(d, ls, dy, dhT, power)
    check(both(d, dy, dhT, cu, power), val, bound)


@pytest.mark.parametrize("lam", [-30.0, -100.0, 0.0, 40.0])
def test_parameters_of_any_size(lam):
    d, dy, dhT, cu, ls = inputs(1, 200, 1, 16, dtype=F32)
    d["lam"] = torch.full((1, 16), lam)
    val, bound = reference(d, ls, dy, dhT)
    # below e^-87 the decay is 1 in fp32, as it is to 30 digits
    if lam == -100.0:
        bound = {k: b + 1e-12 * (1 + val[k].abs()) for k, b in bound.items()}
    check(both(d, dy, dhT, cu), val, bound)


def test_masked_tokens_leave_the_state():
    # a recurrence gate of minus infinity, or the type's lowest value: a = 1, and no gradient passes the token's inputs
    d, dy, dhT, cu, ls = inputs(2, 70, 1, 16)
    d["r"][0, 10:20] = -torch.inf
    d["r"][1, 60:] = torch.finfo(BF).min
    got = both(d, dy, dhT, cu)
    y = got["y"].cpu()
    assert torch.equal(y[0, 10:20], y[0, 9:10].expand(10, -1, -1))
    assert torch.equal(y[1, 60:], y[1, 59:60].expand(10, -1, -1))
    for k in ("dx", "dr", "di"):
        assert not got[k][0, 10:20].any() and not got[k][1, 60:].any(), k
    for k in got:
        assert torch.isfinite(got[k]).all(), k


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_channel_and_sequence(bad):
    lens = [50, 0, 70, 300, 80]
    d, dy, dhT, cu, _ = inputs(1, 500, 1, 72, lens)
    clean = both(d, dy, dhT, cu)
    d["x"][0, 60, 0, 5] = bad       # the third sequence, token 10
    dy[0, 100, 0, 9] = bad
    got = both(d, dy, dhT, cu)
    for k in ("y", "dx", "dr", "di"):
        same = got[k] == clean[k]
        other = torch.ones(72, dtype=torch.bool)
        other[[5, 9]] = False
        assert same[..., other].all(), k
        assert same[0, :50].all() and same[0, 120:].all(), k
    assert torch.equal(got["y"][0, :60], clean["y"][0, :60])
    assert not torch.isfinite(got["y"][0, 60:120, 0, 5]).any()
    keep = [0, 1, 3, 4]
    assert torch.equal(got["hT"][keep], clean["hT"][keep]) and torch.equal(got["dh0"][keep], clean["dh0"][keep])


def test_no_tokens():
    d, dy, dhT, _, _ = inputs(3, 0, 2, 8)
    got = both(d, dy, dhT, None)
    assert got["y"].shape == (3, 0, 2, 8)
    assert torch.equal(got["hT"].cpu(), d["h0"]) and torch.equal(got["dh0"].cpu(), dhT)
    assert not got["dlam"].any() and not got["dbr"].any() and not got["dbi"].any()


@pytest.mark.parametrize("T,lens", [(300, [100, 0, 57]), (300, [0, 0]), (1400, [600, 500]), (64, [64])])
def test_rows_behind_the_last_sequence(T, lens):
    # zero from Python, whatever their inputs hold; and left as they were through the C entries
    d, dy, dhT, cu, ls = inputs(1, T, 1, 24, lens)
    used = sum(lens)
    val, bound = reference(d, ls, dy, dhT)
    for k in ("x", "r", "i"):
        d[k][0, used:] = torch.nan
    dy[0, used:] = torch.inf
    got = both(d, dy, dhT, cu)
    check(got, val, bound)
    for k in ("y", "dx", "dr", "di"):
        assert not got[k][0, used:].any(), k
    c, lib = cuda(d), dn.load_library()
    y = torch.full_like(c["x"], 7.0)
    out = [torch.full_like(c["x"], 7.0) for _ in range(3)]
    ws = torch.empty(lib.dn_glr_bwd_workspace(1, T, 1, 24, 0) + lib.dn_glr_fwd_workspace(1, T, 1, 24) + 16, dtype=torch.uint8, device="cuda")
    dlam = torch.empty_like(c["lam"])
    cu, dy = cu.cuda(), dy.cuda()
    a = lambda t: t.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    ins = [a(c[k]) for k in ("x", "r", "i", "lam", "br", "bi")]
    assert lib.dn_glr_fwd(1, T, 1, 24, len(lens), 1, *ins, 8.0, a(c["h0"]), a(cu), a(y), None, None, a(ws), ws.numel(), st) == 0
    assert lib.dn_glr_bwd(1, T, 1, 24, len(lens), 1, *ins, 8.0, a(c["h0"]), a(cu), None, a(dy), None, *[a(o) for o in out], a(dlam),
                          None, None, None, a(ws), ws.numel(), st) == 0
    torch.cuda.synchronize()
    assert torch.equal(y[0, :used], got["y"][0, :used])
    for t in [y] + out:
        assert (t[0, used:] == 7).all()


def test_continues_in_pieces_and_by_tokens():
    d, _, _, _, ls = inputs(2, 300, 2, 24)
    val, bound = reference(d, ls)
    c = cuda(d)
    cut = lambda a, b: [c[k][:, a:b].contiguous() for k in ("x", "r", "i")]  # noqa: E731
    p = (c["lam"], c["br"], c["bi"])
    y1, h = dn.glr_fwd(*cut(0, 130), *p, c["h0"])
    y2, h = dn.glr_fwd(*cut(130, 280), *p, h)
    ys = [y1, y2]
    for t in range(280, 300):
        ys.append(dn.glr_step(*[a[:, 0] for a in cut(t, t + 1)], *p, h)[:, None])
    check(dict(y=torch.cat(ys, 1), hT=h), val, bound)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,D", [(1, 1, 8), (3, 5, 24), (256, 4, 128)])
def test_step(B, H, D, dtype):
    d, _, _, _, _ = inputs(B, 1, H, D, dtype=dtype)
    val, bound = reference(d, [1] * B)
    c = cuda(d)
    h = c["h0"]
    y = dn.glr_step(c["x"][:, 0], c["r"][:, 0], c["i"][:, 0], c["lam"], c["br"], c["bi"], h)
    check(dict(y=y, hT=h), val, bound)


def test_autograd_and_second_use():
    d, dy, dhT, cu, ls = inputs(1, 200, 2, 16, [120, 80], dtype=F32)
    val, bound = reference(d, ls, dy, dhT)
    c = {k: v.cuda().requires_grad_() for k, v in d.items()}
    for save in (True, False):
        y, hT = dn.glr_scan(*c.values(), cu.cuda(), save_states=save)
        grads = torch.autograd.grad([y, hT], list(c.values()), [dy.cuda(), dhT.cuda()])
        check(dict(zip(("dx", "dr", "di", "dlam", "dbr", "dbi", "dh0"), grads), y=y.detach(), hT=hT.detach()), val, bound)
    # one output alone; a view as gradient
    y, hT = dn.glr_scan(*c.values(), cu.cuda())
    only = torch.autograd.grad(hT.sum(), [c["x"], c["h0"]], retain_graph=True)
    v2, b2 = reference(d, ls, torch.zeros_like(dy), torch.ones_like(dhT))
    check(dict(dx=only[0], dh0=only[1]), v2, b2, ["dx", "dh0"])
    (gx,) = torch.autograd.grad(y.transpose(2, 3).sum(), [c["x"]])
    v3, b3 = reference(d, ls, torch.ones_like(dy), torch.zeros_like(dhT))
    check(dict(dx=gx), v3, b3, ["dx"])


def test_another_stream_and_graph_replays():
    d, dy, dhT, cu, _ = inputs(1, 1500, 1, 136, [700, 0, 300, 500])
    want = both(d, dy, dhT, cu)
    c, dy, dhT, cu = cuda(d), dy.cuda(), dhT.cuda(), cu.cuda()

    def step():
        states = dn.glr_states(c["x"])
        y, hT = dn.glr_fwd(**c, cu_seqlens=cu, states=states)
        return dict(dn.glr_bwd(*c.values(), dy, dhT, cu, states=states), y=y, hT=hT)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x1 = c["x"].clone()
    for n in range(4):
        c["x"].copy_(x1 * (1 + n % 2))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(got[k], eager[k]), (n, k)


@pytest.mark.parametrize("B,T,H,D,lens", [(4, 4096, 4, 128, None), (1, 20000, 2, 128, None), (1, 9000, 1, 1024, [4000, 1, 4999])])
def test_long_sequences_repeat_and_agree(B, T, H, D, lens):
    # against the same kernels on short pieces (within the reference's reach) and bit for bit with themselves
    d, dy, dhT, cu, ls = inputs(B, T, H, D, lens)
    a, b = both(d, dy, dhT, cu), both(d, dy, dhT, cu)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    # channels are independent: a few of them by the reference
    pick = [0, 5, H * D - 1]
    few = {k: v if v is None else v.reshape(*v.shape[:-2], -1)[..., pick][..., None, :] for k, v in d.items()}
    col = lambda v: v.reshape(*v.shape[:-2], -1)[..., pick][..., None, :]  # noqa: E731
    val, bound = reference(few, ls, col(dy), col(dhT))
    check({k: col(v).cpu() for k, v in a.items()}, val, bound)


def test_offsets_past_32_bits():
    # 2^31 + values of x: the last rows' addresses need more than 32 bits
    T, C = 66000, 32768
    x = torch.zeros(1, T, 1, C, dtype=BF, device="cuda")
    x[0, -200:] = 1
    lam = torch.zeros(1, C, device="cuda")
    y, hT = dn.glr_fwd(x, x, x, lam)
    s = torch.sigmoid(torch.tensor(1.0, dtype=torch.float64))
    a = torch.exp(-8 * torch.log(torch.tensor(2.0, dtype=torch.float64)) * s)
    want = torch.sqrt(1 - a * a) * s / (1 - a)
    assert ((hT - want).abs() <= 64 * ref.U * want).all()
    assert not y[0, : T - 200].any() and ((y[0, -1].double() - want).abs() <= ref.half(BF) * want * 1.01).all()


# How a call is cut: one sequence in segments, a pack in segments, a pack and a batch in one walk each,
# short sequences side by side
PLANS = [(1, 4096, 1, 64, None), (1, 1500, 1, 72, [300, 0, 700, 1, 400]), (1, 700, 130, 64, [150, 500, 50]),
         (2, 600, 130, 64, None), (6, 300, 1, 40, None)]


@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("power", [8.0, 1e4])
@pytest.mark.parametrize("B,T,H,D,lens", PLANS)
def test_what_is_not_finite_reaches_its_sequence_under_strong_decays(B, T, H, D, lens, power, bad):
    """Decays whose products (at power 1e4 they themselves) fall below fp32: later tokens, and going back earlier ones,
    still see it, and other sequences and channels do not."""
    d, dy, dhT, cu, ls = inputs(B, T, H, D, lens)
    d["lam"].zero_()
    clean = both(d, dy, dhT, cu, power)
    starts = torch.tensor([0] + ls).cumsum(0)
    n = max(range(len(ls)), key=lambda k: ls[k])  # the longest sequence
    s, e = int(starts[n]), int(starts[n + 1])
    fwd, back = s + min(10, ls[n] // 4), e - 1 - min(7, ls[n] // 4)
    d["x"].reshape(-1, H * D)[fwd, 5] = bad
    dy.reshape(-1, H * D)[back, 9] = bad
    got = both(d, dy, dhT, cu, power)
    flat = lambda t: t.reshape(-1, H * D)  # noqa: E731
    assert not torch.isfinite(flat(got["y"])[fwd:e, 5]).any() and not torch.isfinite(flat(got["hT"])[n, 5])
    assert not torch.isfinite(flat(got["dx"])[s:back + 1, 9]).any() and not torch.isfinite(flat(got["dh0"])[n, 9])
    other = torch.ones(H * D, dtype=torch.bool)
    other[[5, 9]] = False
    for k in ("y", "dx", "dr", "di"):
        same = flat(got[k] == clean[k])
        assert same[:, other].all() and same[:s].all() and same[e:].all(), k
    for k in ("hT", "dh0"):
        same = flat(got[k] == clean[k])
        assert same[:, other].all() and same[:n].all() and same[n + 1:].all(), k
    assert torch.equal(flat(got["y"])[s:fwd], flat(clean["y"])[s:fwd])
    again = both(d, dy, dhT, cu, power, keep=False)
    for k in got:
        assert torch.equal(torch.isfinite(again[k]), torch.isfinite(got[k])), k


@pytest.mark.parametrize("H,lens", [(1, [50, 3, 70, 300, 77]), (130, [50, 3, 70, 300, 77]), (1, [1] * 40 + [200, 0, 260])])
def test_gates_that_are_not_numbers_stay_in_their_sequence(H, lens):
    """A decay of NaN takes no sequence with it that starts, or ends, in the same run of rows."""
    d, dy, dhT, cu, _ = inputs(1, sum(lens), H, 64, lens)
    clean = both(d, dy, dhT, cu)
    starts = [0] + torch.tensor(lens).cumsum(0).tolist()
    hit = [k for k in (1, 2, len(lens) - 3) if lens[k]]
    for n in hit:  # the sequence's first and last tokens
        d["r"][0, [starts[n], starts[n + 1] - 1], 0, 5] = torch.nan
    got = both(d, dy, dhT, cu)
    rows = torch.ones(sum(lens), dtype=torch.bool)
    for n in hit:
        rows[starts[n]:starts[n + 1]] = False
        assert torch.isnan(got["y"][0, starts[n]:starts[n + 1], 0, 5]).all() and torch.isnan(got["hT"][n, 0, 5])
    for k in ("y", "dx", "dr", "di"):
        assert torch.equal(got[k][0, rows.cuda()], clean[k][0, rows.cuda()]), k
    keep = [n for n in range(len(lens)) if n not in hit]
    for k in ("hT", "dh0"):
        assert torch.equal(got[k][keep], clean[k][keep]), k
