"""The 64-bit references of the operators around the token mixers against things
other than themselves (differences, closed forms, published vectors); and the
operators' refusals, which need no GPU."""
import math

import pytest
import torch

import block_ref as ref
import chunkwise_delta_rule_wy_amd as dn

F64 = torch.float64


def gen(*shape, seed=0, scale=1.0):
    return scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def test_recurrence_closed_forms():
    # one channel, constant gates: h_T = a^T h0 + m u (1 - a^T) / (1 - a)
    T, power, lam = 7, 3.0, 0.3
    one = torch.ones(T, 1, dtype=F64)
    val, _ = ref.glr(2 * one, 0.5 * one, -0.25 * one, torch.tensor([lam], dtype=F64), None, None, torch.tensor([[1.5]], dtype=F64), [T],
                     power)
    a = math.exp(-power * math.log1p(math.exp(lam)) / (1 + math.exp(-0.5)))
    u = math.sqrt(1 - a * a) / (1 + math.exp(0.25)) * 2
    assert abs(val["hT"].item() - (a ** T * 1.5 + u * (1 - a ** T) / (1 - a))) < 1e-14
    # a closed recurrence gate keeps the state
    val, _ = ref.glr(one, -torch.inf * one, one, torch.tensor([lam], dtype=F64), None, None, torch.tensor([[1.5]], dtype=F64), [T], power)
    assert (val["y"] == 1.5).all()


def test_recurrence_gradients_against_differences():
    lens, C = [3, 0, 6, 1], 3
    R, N = 12, len(lens)  # two rows behind the last sequence
    x = dict(x=gen(R, C, seed=1), r=gen(R, C, seed=2), i=gen(R, C, seed=3), lam=gen(C, seed=4), br=gen(C, seed=5),
             bi=gen(C, seed=6), h0=gen(N, C, seed=7))
    dy, dhT = gen(R, C, seed=8), gen(N, C, seed=9)
    dy[10:] = 0
    val, _ = ref.glr(**x, lens=lens, power=2.0, dy=dy, dhT=dhT)

    def loss(y):
        v, _ = ref.glr(**y, lens=lens, power=2.0)
        return float((v["y"] * dy).sum() + (v["hT"] * dhT).sum())

    for n, g in dict(x="dx", r="dr", i="di", lam="dlam", br="dbr", bi="dbi", h0="dh0").items():
        d, e = gen(*x[n].shape, seed=20), 1e-6
        diff = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(diff - float((val[g] * d).sum())) < 1e-6 * (1 + abs(diff)), n


def test_norm_gradients_against_differences():
    h, w, dy, dh = gen(3, 8, seed=1), gen(8, seed=2), gen(3, 8, seed=3), gen(3, 8, seed=4)
    _, dres, dw = ref.norm(h, w, 1e-3, dy, dh)
    loss = lambda h, w: float((ref.norm(h, w, 1e-3) * dy).sum() + (h * dh).sum())  # noqa: E731
    for t, g in ((0, dres), (1, dw)):
        d, e = gen(*(h, w)[t].shape, seed=5), 1e-6
        a, b = [h, w], [h, w]
        a[t], b[t] = a[t] + e * d, b[t] - e * d
        assert abs((loss(*a) - loss(*b)) / (2 * e) - float((g * d).sum())) < 1e-7


def test_random_bits():
    # full avalanche: a changed bit of the counter, the stream or the key changes about half of the 128 bits
    base = ref.philox(1, 2, 3)
    for args in ((1, 2, 2), (1, 3, 3), (0, 2, 3), (1, 2, 3 ^ 1 << 40), (1 ^ 1 << 63, 2, 3), (1, 2 ^ 1 << 63, 3)):
        flips = sum(bin(a ^ b).count("1") for a, b in zip(base, ref.philox(*args)))
        assert 34 < flips < 94, (args, flips)  # 64 +- 5.3 deviations of 5.7
    keep = ref.keep_factors([7, 8], 0.25, 40, 200)
    assert set(keep.unique().tolist()) == {0.0, 65536 / 49152}
    assert abs((keep == 0).double().mean().item() - 0.25) < 6 * (0.1875 / 8000) ** 0.5
    assert torch.equal(ref.keep_factors([7, 8], 0.25, 2, 200, 5), keep[5:7])
    assert (ref.keep_factors([7, 8], 1e-6, 2, 200) == 1).all()


# ---------------------------------------------------------------- refusals

F = 0x10000  # aligned, never dereferenced: validation fails first
OK, EINVAL, EUNSUPPORTED, ENOWS = 0, 1, 2, 3
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    return dn.load_library()


def glr_fwd(lib, B=2, T=128, H=4, D=64, n=None, dtype=1, x=F, r=F, i=F, lam=F, power=8.0, h0=None, cu=None, y=F, hT=None,
            states=None, ws=None, wsb=0):
    return lib.dn_glr_fwd(B, T, H, D, B if n is None else n, dtype, x, r, i, lam, None, None, power, h0, cu, y, hT, states,
                          ws, wsb, None)


def glr_bwd(lib, B=2, T=128, H=4, D=64, n=None, dtype=1, dy=F, dx=F, dlam=F, dh0=None, cu=None, states=None, ws=None, wsb=0, power=8.0):
    return lib.dn_glr_bwd(B, T, H, D, B if n is None else n, dtype, F, F, F, F, None, None, power, None, cu, states, dy, None,
                          dx, F, F, dlam, None, None, dh0, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), EINVAL), (dict(T=-1), EINVAL), (dict(H=0), EINVAL), (dict(D=0), EINVAL), (dict(n=3), EINVAL),
    (dict(dtype=2), EINVAL), (dict(cu=F), EINVAL), (dict(power=0.0), EINVAL), (dict(power=-1.0), EINVAL),
    (dict(power=float("nan")), EINVAL), (dict(power=float("inf")), EINVAL), (dict(D=12), EUNSUPPORTED), (dict(D=4), EUNSUPPORTED),
    (dict(H=1 << 20, D=16), EUNSUPPORTED), (dict(H=TOP, D=8), EUNSUPPORTED), (dict(B=1 << 16, T=1 << 15), EUNSUPPORTED),
    (dict(B=TOP, T=TOP), EUNSUPPORTED), (dict(B=1 << 21, T=512, H=1, D=320), EUNSUPPORTED)])
def test_recurrence_refuses_shapes(lib, kw, code):
    assert glr_fwd(lib, **kw) == code
    assert glr_bwd(lib, **kw) == code


def test_recurrence_refuses_pointers_and_workspaces(lib):
    for kw in (dict(x=None), dict(r=None), dict(i=None), dict(lam=None), dict(y=None), dict(x=F + 2), dict(r=F + 8), dict(y=F + 4),
               dict(h0=F + 4), dict(hT=F + 8), dict(states=F + 4)):
        assert glr_fwd(lib, **kw) == EINVAL, kw
    for kw in (dict(dy=None), dict(dx=None), dict(dlam=None), dict(dy=F + 2), dict(dx=F + 8), dict(dh0=F + 4), dict(states=F + 8)):
        assert glr_bwd(lib, **kw) == EINVAL, kw
    # one long sequence is cut into segments, whose maps take memory; the backward pass always sums parameters' gradients
    long = dict(B=1, T=4096)
    need = lib.dn_glr_fwd_workspace(1, 4096, 4, 64)
    assert need > 0 and glr_fwd(lib, **long, ws=F, wsb=need - 1) == ENOWS and glr_fwd(lib, **long) == ENOWS
    assert glr_fwd(lib, **long, ws=F + 8, wsb=need) == ENOWS
    given, none = lib.dn_glr_bwd_workspace(1, 4096, 4, 64, 1), lib.dn_glr_bwd_workspace(1, 4096, 4, 64, 0)
    assert none >= given + 4 * 256 * lib.dn_glr_states(1, 4096, 4, 64)
    assert glr_bwd(lib, **long, states=F, ws=F, wsb=given - 1) == ENOWS and glr_bwd(lib, **long, ws=F, wsb=none - 1) == ENOWS
    assert glr_bwd(lib) == ENOWS


def test_recurrence_sizes_of_memory(lib):
    assert lib.dn_glr_states(1, 1, 1, 8) == 1 and lib.dn_glr_states(3, 65, 1, 8) >= 4
    assert lib.dn_glr_states(2, 640, 1, 8) == 20 and lib.dn_glr_states(1, 0, 1, 8) == 0
    for bad in ((0, 1, 1, 8), (1, -1, 1, 8), (TOP, TOP, 1, 8), (1, 1, TOP, TOP)):
        assert lib.dn_glr_states(*bad) == 0 and lib.dn_glr_fwd_workspace(*bad) == 0 and lib.dn_glr_bwd_workspace(*bad, 0) == 0


@pytest.mark.parametrize("kw,code", [(dict(B=0), EINVAL), (dict(D=12), EUNSUPPORTED), (dict(dtype=3), EINVAL), (dict(dtype=0x101), EINVAL),
                                     (dict(x=None), EINVAL), (dict(state=F + 4), EINVAL), (dict(power=0.0), EINVAL),
                                     (dict(B=1 << 20, H=1 << 14, D=512), EUNSUPPORTED)])
def test_recurrence_step_refuses(lib, kw, code):
    a = dict(B=2, H=1, D=8, dtype=1, x=F, r=F, i=F, lam=F, br=None, bi=None, power=8.0, state=F, y=F, stream=None)
    assert lib.dn_glr_step(*{**a, **kw}.values()) == code


def add_norm(lib, rows=4, D=64, dtype=1, res=1, x=F, residual=F, w=F, p=0.0, seed=None, y=F, h=F):
    return lib.dn_add_norm(rows, D, dtype, res, x, residual, w, 1e-5, p, seed, y, h, None)


def add_norm_bwd(lib, rows=4, D=64, dtype=1, res=1, h=F, w=F, p=0.0, seed=None, dy=F, dh=F, dx=F, dres=F, dw=F, ws=F, wsb=1 << 40):
    return lib.dn_add_norm_bwd(rows, D, dtype, res, h, w, 1e-5, p, seed, dy, dh, dx, dres, dw, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(D=0), EINVAL), (dict(dtype=2), EINVAL), (dict(dtype=0, res=1), EINVAL), (dict(res=3), EINVAL),
    (dict(D=12), EUNSUPPORTED), (dict(D=8200), EUNSUPPORTED), (dict(rows=2 ** 31), EUNSUPPORTED), (dict(w=None), EINVAL),
    (dict(p=1.0, seed=F), EINVAL), (dict(p=-0.1, seed=F), EINVAL), (dict(p=float("nan"), seed=F), EINVAL), (dict(p=0.5), EINVAL),
    (dict(p=1 - 1e-9, seed=F), EUNSUPPORTED), (dict(h=F + 8), EINVAL)])
def test_add_norm_refuses(lib, kw, code):
    assert add_norm(lib, **kw) == code
    assert add_norm_bwd(lib, **kw) == code


def test_add_norm_refuses_pointers_and_workspaces(lib):
    for kw in (dict(x=None), dict(y=None), dict(x=F + 2), dict(residual=F + 4), dict(y=F + 8)):
        assert add_norm(lib, **kw) == EINVAL, kw
    for kw in (dict(h=None), dict(dy=None), dict(dw=None), dict(dy=F + 2), dict(dh=F + 4), dict(dx=F + 8), dict(dres=F + 2)):
        assert add_norm_bwd(lib, **kw) == EINVAL, kw
    need = lib.dn_add_norm_bwd_workspace(4, 64)
    assert need > 0 and add_norm_bwd(lib, wsb=need - 1) == ENOWS and add_norm_bwd(lib, ws=None) == ENOWS
    assert add_norm_bwd(lib, ws=F + 8) == ENOWS
    assert lib.dn_add_norm_bwd_workspace(-1, 64) == lib.dn_add_norm_bwd_workspace(4, 0) == 0
    assert add_norm(lib, rows=0, x=None, y=None) == OK  # nothing to do


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(D=12), EUNSUPPORTED), (dict(dtype=0, res=1), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL),
    (dict(scale=None), EINVAL), (dict(y=F + 8), EINVAL), (dict(x=F + 2), EINVAL), (dict(rows=0, x=None), OK)])
def test_norm8_refuses(lib, kw, code):
    a = dict(rows=4, D=64, dtype=1, res=1, x=F, residual=F, w=F, eps=1e-5, y=F, scale=F, h=F, stream=None)
    assert lib.dn_norm8(*{**a, **kw}.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(act=3), EINVAL), (dict(act=-1), EINVAL), (dict(K=24), EUNSUPPORTED),
    (dict(K=TOP - 15), EUNSUPPORTED), (dict(K=(1 << 23) + 16), EUNSUPPORTED), (dict(M=TOP), EUNSUPPORTED), (dict(N=TOP), EUNSUPPORTED), (dict(M=1 << 20, N=1 << 20), EUNSUPPORTED),
    (dict(x=None), EINVAL), (dict(xs=None), EINVAL), (dict(w=None), EINVAL), (dict(ws=None), EINVAL), (dict(y=None), EINVAL),
    (dict(x=F + 8), EINVAL), (dict(w=F + 8), EINVAL), (dict(residual=F + 2), EINVAL), (dict(y=F + 2), EINVAL), (dict(M=0, x=None), OK)])
def test_linear8_refuses(lib, kw, code):
    a = dict(M=4, N=64, K=64, x=F, xs=F, w=F, ws=F, bias=None, residual=None, act=0, y=F, stream=None)
    assert lib.dn_linear8(*{**a, **kw}.values()) == code


@pytest.mark.parametrize("M", [1, 64, 65])
def test_linear8_refuses_grids_of_too_many_threads(lib, M):
    assert lib.dn_linear8(M, (1 << 26) + 1, 64, F, F, F, F, None, None, 0, F, None) == EUNSUPPORTED


def test_python_refuses():
    x, w = torch.zeros(2, 3, 1, 8), torch.zeros(1, 8)
    for call in (lambda: dn.glr_fwd(x, x, x, w), lambda: dn.glr_bwd(x, x, x, w, None, None, None, x), lambda: dn.glr_scan(x, x, x, w),
                 lambda: dn.glr_step(x[:, 0], x[:, 0], x[:, 0], w, None, None, x[:, 0]), lambda: dn.glr_states(x),
                 lambda: dn.add_norm(x, x, w[0]), lambda: dn.add_norm_bwd(x, w[0], x), lambda: dn.add_norm_fn(x, None, w[0]),
                 lambda: dn.norm8(x),
                 lambda: dn.linear8(x.to(torch.float8_e4m3fn), w, w.to(torch.float8_e4m3fn), w)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        dn.glr_fwd(x.half(), x, x, w)
    with pytest.raises(TypeError):
        dn.linear8(x, w, x, w)
    with pytest.raises(ValueError, match="act"):
        dn.linear8(x, w, x, w, act="relu")
    with pytest.raises(ValueError, match="dimensions"):
        dn.glr_fwd(x[0], x, x, w)


def test_random_bits_against_published_vectors():
    # the known answers that the method's authors publish for 4 words and 7 rounds (Salmon et al., 2011): counters and
    # keys of zeros, of ones, and of the digits of pi
    cases = [(0, 0, 0, "5f6fb709 0d893f64 4f121f81 4f730a48"),
             (2 ** 64 - 1, 2 ** 64 - 1, 2 ** 64 - 1, "5207ddc2 45165e59 4d8ee751 8c52f662"),
             (0x299F31D0A4093822, 0x0370734413198A2E, 0x85A308D3243F6A88, "4dfccaba 190a87f0 c47362ba b6b5242a")]
    for key, stream, block, want in cases:
        assert ref.philox(key, stream, block) == [int(v, 16) for v in want.split()]
