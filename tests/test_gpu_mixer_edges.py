"""The state space mixer's operators where calls meet: the two directions of a
cut backward pass, packs that end before their rows do, many short sequences,
and the fp32 accuracy of states and parameter gradients."""
import ctypes

import pytest
import torch

import chunkwise_delta_rule_wy_amd as dn
import mixer_ref as ref
from test_gpu_mixer import BF, F32, cu_of, cuda, randn, reference, scan_inputs

pytestmark = pytest.mark.gpu


def test_segment_decays_have_one_writer():
    """The backward pass's first sweeps run both ways at once.  A segment's log decay is the sum that
    the forward order gives, bit for bit the forward pass's (whose packed plan is the same), and
    only a last segment's comes from the reverse sweep.  The sums lie in the workspace behind the
    packed tables: the segments' bases and sequences and, backwards, the chunks' as well."""
    lens, H, G, dk, dv = [1500, 0, 1100], 4, 1, 64, 64
    T, N = sum(lens), len(lens)
    seg, up = 256, lambda n: (n + 255) // 256 * 256  # tokens of a segment: four chunks
    nseg, nchunks = T // seg + N, T // 64 + N
    x, dO, dhT, _ = scan_inputs(1, T, H, G, dk, dv, lens)
    d, cu, dO, dhT = cuda(x), cu_of(lens), dO.cuda(), dhT.cuda()
    lib, s = dn.load_library(), ctypes.byref(dn._SsmShape(1, T, H, G, dk, dv, N, 1))
    p = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    ins = p(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], cu)
    st = torch.cuda.current_stream().cuda_stream
    out = [torch.empty_like(d[n]) for n in ("v", "h0")]
    gr = [torch.empty_like(d[n]) for n in ("q", "k", "v", "dt", "A", "A", "A", "h0")]
    ws = [torch.full((f(s),), 255, dtype=torch.uint8, device="cuda") for f in (lib.dn_ssm_fwd_workspace, lib.dn_ssm_bwd_workspace)]
    assert lib.dn_ssm_fwd(s, *ins, *p(*out), ws[0].data_ptr(), ws[0].numel(), st) == 0
    assert lib.dn_ssm_bwd(s, *ins, *p(dO, dhT, *gr), ws[1].data_ptr(), ws[1].numel(), st) == 0
    at = [up(4 * (N + 1 + nseg)), up(4 * (N + 1 + nseg + N + 1 + nchunks))]
    fwd, bwd = (w[a:a + 8 * nseg * H].view(torch.float64).view(nseg, H).cpu() for w, a in zip(ws, at))
    per = [(n + seg - 1) // seg for n in lens]
    last = [sum(per[:i + 1]) - 1 for i in range(N) if per[i]]
    inner = [i for i in range(sum(per)) if i not in last]
    assert len(inner) == 9 and (fwd[inner] < 0).all() and torch.isfinite(fwd[inner]).all()
    assert torch.equal(fwd[inner], bwd[inner])
    assert torch.isnan(fwd[last]).all() and (bwd[last] < 0).all()


def padded(t, tail):
    """Rows of NaN behind the tokens of a [1,T,...] tensor."""
    return torch.cat([t, torch.full((1, tail, *t.shape[2:]), float("nan"), dtype=t.dtype, device=t.device)], 1)


def spoil_free_memory(total=1 << 28):
    """Leaves NaN in the memory that the next tensors get."""
    for size in (1 << 12, 1 << 14, 1 << 16, 1 << 18, 1 << 20, 1 << 22):
        junk = [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(min(64, total // size))]
        del junk


@pytest.mark.parametrize("lens,tail,H,G,dk,dv", [
    ([70, 0, 33], 97, 4, 1, 64, 64),        # whole chunks behind the last sequence
    ([2200, 5], 100, 2, 1, 64, 64),         # cut into segments
    ([64, 63], 1, 3, 3, 64, 128),           # one row
    ([0, 0], 40, 4, 2, 64, 64),             # no tokens at all
    ([5], 0, 2, 1, 64, 64),                 # no rows behind
    ([130], 4000, 1, 1, 128, 64),           # few workgroups, many rows
])
def test_rows_behind_the_last_sequence_are_zero(lens, tail, H, G, dk, dv):
    """Where offsets end before the rows do, the Python functions return zeros there, whatever the
    rows hold, and everything before them as without the rows."""
    n = sum(lens)
    x, dO, dhT, _ = scan_inputs(1, n, H, G, dk, dv, lens)
    d, cu, dO, dhT = cuda(x), cu_of(lens), dO.cuda(), dhT.cuda()
    w, b = randn(H, dv, 4, seed=21).cuda(), randn(H, dv, seed=22).cuda()
    s0 = randn(len(lens), 3, H, dv, seed=23, dtype=BF).cuda()

    def calls(d, dO):
        par = (d["A"], d["dt_bias"], d["skip"], d["h0"])
        spoil_free_memory()
        o, hT = dn.ssm_fwd(d["q"], d["k"], d["v"], d["dt"], *par, cu)
        spoil_free_memory()
        g = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], *par, dO, dhT, cu)
        spoil_free_memory()
        y, sT = dn.conv_silu(d["v"], w, b, s0, cu)
        spoil_free_memory()
        gc = dn.conv_silu_bwd(d["v"], w, b, s0, dO, s0, cu)
        return dict(g, o=o, hT=hT, y=y, sT=sT, **{"conv_" + k: t for k, t in gc.items()})

    want = calls(d, dO)
    got = calls({k: padded(t, tail) if k in ("q", "k", "v", "dt") else t for k, t in d.items()}, padded(dO, tail))
    # the plan of a longer tensor may cut elsewhere: compared bit for bit where it does not
    val, bound = reference(x, lens, dO.cpu(), dhT.cpu())
    for name, t in got.items():
        if t.shape[:2] == (1, n + tail):
            assert not t[:, n:].any(), name  # NaN counts as any
            got[name] = t = t[:, :n]
        if name in val:
            assert ref.worst(t.reshape(val[name].shape), val[name], bound[name]) <= 1, name
        elif name not in ("conv_dw", "conv_dbias"):
            assert torch.equal(t, want[name]), name
        else:  # the same terms |dz x|, |dz| <= 1.1 |dy|, added in two orders
            terms = 1.1 * dO.float().abs().sum(1) * max([1.0] + [float(t.abs().max()) for t in (d["v"], s0) if t.numel()])
            terms = terms[0] if name == "conv_dbias" else terms[0, ..., None]
            assert ((t - want[name]).abs() <= 2 * (n + 64) * ref.U32 * terms).all(), name


@pytest.mark.parametrize("lens,tail", [([40, 0, 110], 75), ([150], 300)])
def test_mixer_trains_on_padded_packs(lens, tail):
    """Projection, convolutions, scan and norm through autograd with rows behind the last sequence:
    the weights' gradients are those of the pack without them, and no gradient holds what the
    memory held before."""
    n, H, G, dk, dv, W = sum(lens), 4, 2, 64, 64, 4
    cu = cu_of(lens)
    par = dict(scale=1 + randn(H, dv, seed=1, scale=0.1), wv=randn(H, dv, W, seed=2, scale=0.5),
               wq=randn(G, dk, W, seed=3, scale=0.5), wk=randn(G, dk, W, seed=4, scale=0.5), bv=randn(H, dv, seed=5),
               A=-1 - randn(H, seed=6).abs(), dt_bias=randn(H, seed=7) - 3, skip=randn(H, seed=8), wn=randn(dv, seed=9))
    data = dict(xv=randn(1, n + tail, H, dv, seed=10), xq=randn(1, n + tail, G, dk, seed=11, dtype=BF),
                xk=randn(1, n + tail, G, dk, seed=12, dtype=BF), dt=randn(1, n + tail, H, seed=13),
                z=randn(1, n + tail, H, dv, seed=14, dtype=BF), weight=randn(1, n + tail, H, dv, seed=15))

    def train(rows):
        p = {k: t.cuda().requires_grad_() for k, t in par.items()}
        x = {k: t[:, :rows].contiguous().cuda().requires_grad_(k != "weight") for k, t in data.items()}
        scaled = x["xv"] * p["scale"]  # stands for the projection, whose weights all rows enter
        spoil_free_memory()
        v, _ = dn.conv_silu_fn(scaled.to(BF), p["wv"], p["bv"], None, cu)
        spoil_free_memory()
        q, _ = dn.conv_silu_fn(x["xq"], p["wq"], None, None, cu)
        k, _ = dn.conv_silu_fn(x["xk"], p["wk"], None, None, cu)
        spoil_free_memory()
        o, _ = dn.ssm_scan(q, k, v, x["dt"], p["A"], p["dt_bias"], p["skip"], None, cu)
        y = dn.gated_norm_fn(o, x["z"], p["wn"])
        kept = dict(scaled=scaled, q=q, k=k, v=v)
        for t in kept.values():
            t.retain_grad()
        spoil_free_memory()
        (y[:, :n].float() * x["weight"][:, :n]).sum().backward()  # a program's loss takes the tokens alone
        # sums of the absolute values of the terms of each sum over tokens (|dz| <= 1.1 |dy|)
        size = {"w" + i: 1.1 * kept[i].grad.float().abs().sum((0, 1))[..., None] * t.float().abs().max()
                for i, t in (("v", scaled), ("q", x["xq"]), ("k", x["xk"]))}
        size.update(bv=1.1 * v.grad.float().abs().sum((0, 1)), scale=(scaled.grad * x["xv"]).abs().sum((0, 1)),
                    wn=(x["weight"][:, :n] * y[:, :n].float() / p["wn"]).abs().sum((0, 1, 2)))
        return {k: t.grad for k, t in x.items() if k != "weight"}, {k: t.grad for k, t in p.items()}, size

    gx, want, size = train(n)
    gx2, got, _ = train(n + tail)
    for name, t in gx2.items():
        assert not t[:, n:].any() and torch.equal(t[:, :n], gx[name]), name
    for name, t in got.items():
        # the same terms, for some parameters added in two orders (the norm's are n H)
        bound = 2 * (n * H + 64) * ref.U32 * size[name].detach() if name in size else 0
        assert torch.isfinite(t).all() and ((t - want[name]).abs() <= bound).all(), name


@pytest.mark.parametrize("T,H,G,dk,dv,rate,bias", [(1100, 4, 2, 128, 64, 1.0, -3.0), (2300, 2, 1, 64, 64, 0.02, -2.0),
                                                   (2048, 8, 1, 128, 128, 0.3, -3.0)])
def test_states_and_parameter_gradients_have_fp32_accuracy(T, H, G, dk, dv, rate, bias):
    """hT, dh0 and the gradients in fp32 against 64 bits over many chunks, uncut and cut, strong and
    weak decays, in the Euclidean norm, which tells three bf16 parts of an fp32 operand from two
    where a bound on the largest error cannot.

    A state is a sum of products with independent relative errors, in half steps of fp32 (U32): the
    step size about 2 (6 at most), the exponents' rounding |x| ln 2 / 2 with |x| below 5 where a weight
    counts, 1.7, the exponential and a product 1.2, and its own sums, six a chunk over the 16 chunks that
    it remembers at the most, each 0.6 on average, 6: the root of their squares is below 7, and 8 is
    asked.  Measured: 1.2 to 2.6; with two parts 15 to 42.

    The parameters' gradients add the tokens' errors up; the independent ones average out, and 6 is
    asked of the sum (whose terms do not cancel for these inputs).  Measured: 0.5 to 2.3; with two
    parts 11 to 82 for dA and ddt_bias, and without the accumulators' change of sign dA 3.2, 12.6, 12.7."""
    g = torch.Generator("cuda").manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    silu = torch.nn.functional.silu
    q, k, v = (silu(n(1, T, *s)).to(BF) for s in ((G, dk), (G, dk), (H, dv)))
    dt, A = n(1, T, H), -rate * (1 + torch.rand(H, generator=g, device="cuda"))
    par = (n(H) * 0.3 + bias, n(H), n(1, H, dk, dv))  # dt_bias, skip, h0
    dO, dhT = n(1, T, H, dv).to(BF), n(1, H, dk, dv)
    leaves = [t.double().requires_grad_() for t in (q, k, v, dt, A, *par)]
    s = ref.softplus(leaves[3][0] + leaves[5])
    o, hT = ref.scan(leaves[0][0], leaves[1][0], leaves[2][0], s, s * leaves[4], leaves[6], leaves[7], [T])
    grads = torch.autograd.grad([o, hT], leaves[3:], [dO[0].double(), dhT.double()])
    want = dict(zip(("ddt", "dA", "ddt_bias", "dskip", "dh0"), grads), hT=hT.detach())
    _, got_h = dn.ssm_fwd(q, k, v, dt, A, *par)
    got = dict(dn.ssm_bwd(q, k, v, dt, A, *par, dO, dhT), hT=got_h)
    for name, limit in dict(hT=8, dh0=8, ddt=8, dA=6, ddt_bias=6, dskip=6).items():
        err = float((got[name].double() - want[name]).norm() / want[name].norm()) / ref.U32
        assert err <= limit, (name, err)


@pytest.mark.parametrize("N,top,H,G,dk,dv,tail", [(150, 60, 2, 1, 64, 64, 0), (300, 20, 3, 3, 64, 128, 65), (40, 130, 4, 1, 128, 64, 7)])
def test_packs_of_many_short_sequences(N, top, H, G, dk, dv, tail):
    """Tens to hundreds of sequences, shorter than a segment and mostly than a chunk, empty ones among
    them, in packs long enough to be cut."""
    gen = torch.Generator().manual_seed(N)
    lens = torch.randint(0, top, (N,), generator=gen).tolist()
    n = sum(lens)
    assert n > 32 * 64
    x, dO, dhT, _ = scan_inputs(1, n, H, G, dk, dv, lens)
    val, bound = reference(x, lens, dO, dhT)
    d = {k: padded(t, tail) if k in ("q", "k", "v", "dt") else t for k, t in cuda(x).items()}
    cu = cu_of(lens)
    o, hT = dn.ssm_fwd(**d, cu_seqlens=cu)
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], padded(dO, tail).cuda(),
                    dhT.cuda(), cu)
    got = dict(gr, o=o, hT=hT)
    for name in val:
        t = got[name]
        if t.shape[:2] == (1, n + tail):
            assert not t[:, n:].any(), name
            t = t[:, :n]
        assert ref.worst(t.reshape(val[name].shape), val[name], bound[name]) <= 1, name


def test_scan_with_growing_states():
    # A > 0 is allowed: the states grow as the formula says
    x, dO, dhT, ls = scan_inputs(1, 300, 2, 1, 64, 64, A=0.05)
    val, bound = reference(x, ls, dO, dhT)
    d = cuda(x)
    o, hT = dn.ssm_fwd(**d)
    gr = dn.ssm_bwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"], dO.cuda(), dhT.cuda())
    for name, t in dict(gr, o=o, hT=hT).items():
        assert ref.worst(t.reshape(val[name].shape), val[name], bound[name]) <= 1, name


def test_captured_passes_follow_the_offsets():
    """Offsets changed between the replays of a captured pass, also to fewer tokens: every replay as
    the eager calls, with zeros behind the sequences where earlier replays left values."""
    T, N, H, G, dk, dv = 2500, 4, 2, 1, 64, 64
    x, dO, dhT, _ = scan_inputs(1, T, H, G, dk, dv, [T - 3, 1, 1, 1])
    d, dO, dhT = cuda(x), dO.cuda(), dhT.cuda()
    w, b = randn(H, dv, 4, seed=1).cuda(), randn(H, dv, seed=2).cuda()
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")

    def train():
        v, sT = dn.conv_silu(d["v"], w, b, None, cu)
        args = (d["q"], d["k"], v, d["dt"], d["A"], d["dt_bias"], d["skip"], d["h0"])
        o, hT = dn.ssm_fwd(*args, cu)
        g = dn.ssm_bwd(*args, dO, dhT, cu)
        gc = dn.conv_silu_bwd(d["v"], w, b, None, g["dv"], None, cu)
        return [v, sT, o, hT, *g.values(), *gc.values()]

    packs = [[2200, 0, 37, 200], [0, 0, 0, 0], [600, 600, 1, 1299], [5, 64, 0, 900], [T, 0, 0, 0]]
    cu.copy_(cu_of(packs[0]))
    train()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train()
    for lens in packs:
        cu.copy_(cu_of(lens))
        graph.replay()
        torch.cuda.synchronize()
        want = train()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), lens
        for t in out:
            if t.shape[:2] == (1, T):
                assert torch.isfinite(t.float()).all() and not t[:, sum(lens):].any()
