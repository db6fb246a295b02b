"""The mixer operators' 64-bit reference against things other than itself:
closed forms, explicit products, central differences; and the operators'
refusals, which need no GPU."""
import ctypes
import math

import pytest
import torch

import chunkwise_delta_rule_wy_amd as dn
import mixer_ref as ref

F64 = torch.float64


def gen(*shape, seed=0, scale=1.0):
    return scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def test_scan_matches_explicit_sums():
    T, H, G, dk, dv = 6, 4, 2, 3, 2
    q, k, v = gen(T, G, dk, seed=1), gen(T, G, dk, seed=2), gen(T, H, dv, seed=3)
    s, a, skip, h0 = gen(T, H, seed=4).abs(), -gen(T, H, seed=5).abs(), gen(H, seed=6), gen(1, H, dk, dv, seed=7)
    o, hT = ref.scan(q, k, v, s, a, skip, h0, [T])
    for h in range(H):
        g = h // 2
        for t in range(T):
            want = skip[h] * v[t, h] + math.exp(a[:t + 1, h].sum()) * (h0[0, h].T @ q[t, g])
            for j in range(t + 1):
                want = want + math.exp(a[j + 1:t + 1, h].sum()) * s[j, h] * (k[j, g] @ q[t, g]) * v[j, h]
            assert torch.allclose(o[t, h], want, rtol=1e-12, atol=1e-12)
    want = math.exp(a[:, 0].sum()) * h0[0, 0] + sum(
        math.exp(a[j + 1:, 0].sum()) * s[j, 0] * torch.outer(k[j, 0], v[j, 0]) for j in range(T))
    assert torch.allclose(hT[0, 0], want, rtol=1e-12, atol=1e-12)


def test_scan_without_decay_is_linear_attention():
    T, dk, dv = 9, 4, 3
    q, k, v = gen(T, 1, dk, seed=1), gen(T, 1, dk, seed=2), gen(T, 1, dv, seed=3)
    o, _ = ref.scan(q, k, v, torch.ones(T, 1, dtype=F64), torch.zeros(T, 1, dtype=F64), torch.zeros(1, dtype=F64),
                    torch.zeros(1, 1, dk, dv, dtype=F64), [T])
    assert torch.allclose(o[:, 0], torch.tril(q[:, 0] @ k[:, 0].T) @ v[:, 0], rtol=1e-12)


def test_scan_gradients_against_differences():
    lens, H, G, dk, dv = [3, 0, 4, 1], 4, 2, 3, 2
    T, N = sum(lens), len(lens)
    x = dict(q=gen(T, G, dk, seed=1), k=gen(T, G, dk, seed=2), v=gen(T, H, dv, seed=3), dt=gen(T, H, seed=4),
             A=-1 - gen(H, seed=5).abs(), bias=gen(H, seed=6), skip=gen(H, seed=7), h0=gen(N, H, dk, dv, seed=8))
    dO, dhT = gen(T, H, dv, seed=9), gen(N, H, dk, dv, seed=10)
    val, _ = ref.scan_with_bounds(**x, lens=lens, dO=dO, dhT=dhT)

    def loss(y):
        s = ref.softplus(y["dt"] + y["bias"])
        o, hT = ref.scan(y["q"], y["k"], y["v"], s, s * y["A"], y["skip"], y["h0"], lens)
        return float((o * dO).sum() + (hT * dhT).sum())

    names = dict(q="dq", k="dk", v="dv", dt="ddt", A="dA", bias="ddt_bias", skip="dskip", h0="dh0")
    for n, g in names.items():
        d, e = gen(*x[n].shape, seed=20), 1e-6
        diff = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(diff - float((val[g] * d).sum())) < 1e-6 * (1 + abs(diff)), n


def test_conv_and_norm_closed_forms():
    x, w = gen(5, 1, 2, seed=1), torch.zeros(1, 2, 3, dtype=F64)
    w[:, :, 2] = 1.0  # only the current token: y = silu(x)
    y, sT = ref.conv_silu(x, w, torch.zeros(1, 2, dtype=F64), gen(1, 2, 1, 2, seed=2), [5])
    assert torch.allclose(y, torch.nn.functional.silu(x)) and torch.equal(sT[0], x[3:])
    u = torch.full((2, 4), 3.0, dtype=F64)
    assert torch.allclose(ref.gated_norm(u, u, torch.ones(4, dtype=F64), 0.0, True), torch.ones(2, 4, dtype=F64))
    want = torch.nn.functional.silu(u)
    assert torch.allclose(ref.gated_norm(u, u, torch.ones(4, dtype=F64), 0.0, False), want)


# ---------------------------------------------------------------- refusals

FAKE = 0x10000  # aligned, never dereferenced: validation fails first
OK, EINVAL, EUNSUPPORTED, ENOWS = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return dn.load_library()


def P(x):
    return ctypes.c_void_p(x)


def ssm_shape(**kw):
    d = dict(B=2, T=128, H=4, G=2, Dk=64, Dv=64, n_seqs=2, dtype=1)
    d.update(kw)
    return dn._SsmShape(**d)


def ssm_fwd(lib, s, q=FAKE, v=FAKE, A=FAKE, o=FAKE, h0=None, cu=None, ws=FAKE, wsb=1 << 40):
    return lib.dn_ssm_fwd(ctypes.byref(s), P(q), P(FAKE), P(v), P(FAKE), P(A), None, None, P(h0), P(cu), P(o), None,
                          P(ws), wsb, None)


def ssm_bwd(lib, s, dO=FAKE, dA=FAKE, dq=FAKE, ws=FAKE, wsb=1 << 50):
    return lib.dn_ssm_bwd(ctypes.byref(s), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, None, None, None, P(dO),
                          None, P(dq), P(FAKE), P(FAKE), P(FAKE), P(dA), None, None, None, P(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), EINVAL), (dict(T=-1), EINVAL), (dict(H=0), EINVAL), (dict(G=0), EINVAL), (dict(G=3), EINVAL),
    (dict(Dk=0), EINVAL), (dict(dtype=5), EINVAL), (dict(n_seqs=3), EINVAL), (dict(Dk=96), EUNSUPPORTED),
    (dict(Dk=256), EUNSUPPORTED), (dict(Dv=48), EUNSUPPORTED), (dict(Dv=2048), EUNSUPPORTED),
    (dict(dtype=0), EUNSUPPORTED), (dict(B=1 << 20, n_seqs=1 << 20, H=4096, G=4096), EUNSUPPORTED),
])
def test_scan_refuses_shapes(lib, kw, code):
    assert ssm_fwd(lib, ssm_shape(**kw)) == code
    assert ssm_bwd(lib, ssm_shape(**kw)) == code


def test_scan_refuses_pointers_and_workspaces(lib):
    s = ssm_shape()
    assert ssm_fwd(lib, s, q=None) == EINVAL and ssm_fwd(lib, s, A=None) == EINVAL
    assert ssm_fwd(lib, s, v=FAKE + 2) == EINVAL and ssm_fwd(lib, s, o=FAKE + 8) == EINVAL
    assert ssm_fwd(lib, s, h0=FAKE + 4) == EINVAL
    assert ssm_fwd(lib, s, cu=FAKE) == EINVAL  # packed input needs B == 1
    assert ssm_bwd(lib, s, dO=None) == EINVAL and ssm_bwd(lib, s, dA=None) == EINVAL
    assert ssm_bwd(lib, s, dq=FAKE + 2) == EINVAL
    need = lib.dn_ssm_bwd_workspace(ctypes.byref(s))
    # two states of 64 x 64 floats for each of 4 chunks and 4 heads at the least
    assert need >= 2 * 4 * 4 * 64 * 64 * 4
    assert ssm_bwd(lib, s, wsb=need - 1) == ENOWS and ssm_bwd(lib, s, ws=None) == ENOWS
    assert ssm_bwd(lib, s, ws=FAKE + 8) == ENOWS
    packed = ssm_shape(B=1, T=4096, n_seqs=5)  # cut into segments, whose states take memory
    need = lib.dn_ssm_fwd_workspace(ctypes.byref(packed))
    assert need > 0 and ssm_fwd(lib, packed, cu=FAKE, wsb=need - 1) == ENOWS
    assert lib.dn_ssm_fwd_workspace(ctypes.byref(ssm_shape(T=10 ** 5, H=400, G=400))) == 0  # streams enough: not cut
    assert lib.dn_ssm_fwd_workspace(ctypes.byref(ssm_shape(B=1, T=2048, n_seqs=9))) == 0  # 32 chunks: not cut


@pytest.mark.parametrize("H,G,Dk,Dv,dtype,state,code", [
    (4, 3, 64, 64, 0, FAKE, EINVAL), (4, 2, 64, 64, 3, FAKE, EINVAL), (4, 2, 80, 64, 0, FAKE, EUNSUPPORTED),
    (4, 2, 64, 96, 1, FAKE, EUNSUPPORTED), (4, 2, 64, 64, 1, None, EINVAL), (4, 2, 64, 64, 1, FAKE + 4, EINVAL)])
def test_step_refuses(lib, H, G, Dk, Dv, dtype, state, code):
    assert lib.dn_ssm_step(2, H, G, Dk, Dv, dtype, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, None, P(state),
                           P(FAKE), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), EINVAL), (dict(T=-1), EINVAL), (dict(D=12), EUNSUPPORTED), (dict(W=0), EUNSUPPORTED),
    (dict(W=5), EUNSUPPORTED), (dict(dtype=2), EINVAL), (dict(n=3), EINVAL), (dict(x=None), EINVAL),
    (dict(x=FAKE + 2), EINVAL), (dict(w=None), EINVAL), (dict(s0=FAKE + 4), EINVAL)])
def test_conv_silu_refuses(lib, kw, code):
    d = dict(B=2, T=8, H=2, D=16, W=4, n=2, dtype=1, x=FAKE, w=FAKE, s0=None)
    d.update(kw)
    dims = [d[i] for i in ("B", "T", "H", "D", "W", "n", "dtype")]
    assert lib.dn_conv_silu(*dims, P(d["x"]), P(d["w"]), None, P(d["s0"]), None, P(FAKE), None, None) == code
    assert lib.dn_conv_silu_bwd(*dims, P(d["x"]), P(d["w"]), None, P(d["s0"]), None, P(FAKE), None, P(FAKE), P(FAKE),
                                None, None, P(FAKE), 1 << 40, None) == code
    if code == EINVAL and not {"T", "n"} & set(kw):
        assert lib.dn_conv_silu_step(d["B"], d["H"], d["D"], d["W"], d["dtype"], P(d["x"]), P(d["w"]), None,
                                     P(d["s0"]), P(FAKE), None) == code


def test_conv_silu_bwd_refuses_workspace(lib):
    need = lib.dn_conv_silu_bwd_workspace(2, 8, 2, 16, 4)
    assert need == 4 * 2 * 16 * 5
    args = [2, 8, 2, 16, 4, 2, 1, P(FAKE), P(FAKE), None, None, None, P(FAKE), None, P(FAKE), P(FAKE), None, None]
    assert lib.dn_conv_silu_bwd(*args, P(FAKE), need - 1, None) == ENOWS
    assert lib.dn_conv_silu_bwd(*args, None, need, None) == ENOWS


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(D=0), EINVAL), (dict(R=0), EINVAL), (dict(rows=7, R=2), EINVAL),
    (dict(dtype=4), EINVAL), (dict(D=20), EUNSUPPORTED), (dict(D=8200), EUNSUPPORTED), (dict(x=None), EINVAL),
    (dict(x=FAKE + 8), EINVAL), (dict(w=None), EINVAL), (dict(rows=1 << 31), EUNSUPPORTED)])
def test_gated_norm_refuses(lib, kw, code):
    d = dict(rows=8, D=64, R=1, dtype=1, x=FAKE, w=FAKE)
    d.update(kw)
    dims = [d[i] for i in ("rows", "D", "R", "dtype")]
    assert lib.dn_gated_norm(*dims, P(d["x"]), P(FAKE), P(d["w"]), 1e-5, 0, P(FAKE), None) == code
    assert lib.dn_gated_norm_bwd(*dims, P(d["x"]), P(FAKE), P(d["w"]), 1e-5, 0, P(FAKE), P(FAKE), P(FAKE), P(FAKE),
                                 P(FAKE), 1 << 40, None) == code


def test_python_refuses_host_tensors_and_types():
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        dn.gated_norm(x, x, torch.ones(64))
    with pytest.raises(ValueError):
        dn.conv_silu(x, torch.zeros(2, 64, 4))
    with pytest.raises(TypeError):
        dn.ssm_fwd(x, x, x, torch.zeros(1, 4, 2), -torch.ones(2))  # float32 chunks are not there
    with pytest.raises(ValueError):
        dn.ssm_step(x[0], x[0], x[0], torch.zeros(4, 2), -torch.ones(2), None, None, torch.zeros(4, 2, 64, 64))


def test_python_refuses_what_is_no_tensor():
    x, w = torch.zeros(2, 2, 64), torch.zeros(2, 64, 4)
    for call in (lambda: dn.ssm_step(None, x, x, x, x, None, None, x), lambda: dn.ssm_step(x, x, None, x, x, None, None, x),
                 lambda: dn.conv_silu_step(None, w, None, x), lambda: dn.conv_silu_step(x, None, None, x),
                 lambda: dn.conv_silu_step(x, w, None, None), lambda: dn.gated_norm(None, x, x),
                 lambda: dn.gated_norm(x, x, None), lambda: dn.gated_norm_bwd(x, None, x, x),
                 lambda: dn.ssm_fwd(None, x, x, x, x), lambda: dn.conv_silu(None, w)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_launches_that_are_too_large_are_refused(lib):
    # 2^20 sequences of 64 heads: 2^26 workgroups of 256 threads are more than a grid has
    assert lib.dn_ssm_step(1 << 20, 64, 1, 64, 64, 1, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, None, P(FAKE),
                           P(FAKE), None) == EUNSUPPORTED
    s = ssm_shape(B=1 << 18, n_seqs=1 << 18, H=64, G=1)
    assert ssm_fwd(lib, s) == EUNSUPPORTED and ssm_bwd(lib, s) == EUNSUPPORTED
    assert ssm_fwd(lib, ssm_shape(H=1 << 18, G=1 << 18, Dv=1024)) == EUNSUPPORTED  # 2^31 bytes between 64 rows
    # 2^27 channels of 16 weights and a bias, and 2^31 channel quadruples times runs
    assert lib.dn_conv_silu(1, 1, 1 << 20, 1 << 9, 4, 1, 1, P(FAKE), P(FAKE), None, None, None, P(FAKE), None,
                            None) == EUNSUPPORTED
    assert lib.dn_conv_silu_bwd_workspace(1, 1, 1 << 20, 1 << 9, 4) == 0
    assert lib.dn_conv_silu(1 << 15, 1 << 15, 8, 64, 4, 1 << 15, 1, P(FAKE), P(FAKE), None, None, None, P(FAKE), None,
                            None) == EUNSUPPORTED


def test_conv_silu_refuses_unaligned_weights(lib):
    for w, b in ((FAKE + 4, FAKE), (FAKE, FAKE + 8)):
        assert lib.dn_conv_silu(1, 4, 1, 8, 4, 1, 1, P(FAKE), P(w), P(b), None, None, P(FAKE), None, None) == EINVAL
        assert lib.dn_conv_silu_step(1, 1, 8, 4, 1, P(FAKE), P(w), P(b), P(FAKE), P(FAKE), None) == EINVAL
        assert lib.dn_conv_silu_bwd(1, 4, 1, 8, 4, 1, 1, P(FAKE), P(w), P(b), None, None, P(FAKE), None, P(FAKE), P(FAKE),
                                    None, None, P(FAKE), 1 << 30, None) == EINVAL


def test_the_tail_flag_belongs_to_packed_passes(lib):
    # accepted with a type, refused without a known one and in calls that know no packs
    assert ssm_fwd(lib, ssm_shape(dtype=0x101), q=None) == EINVAL
    assert ssm_fwd(lib, ssm_shape(dtype=0x100)) == EUNSUPPORTED and ssm_fwd(lib, ssm_shape(dtype=0x105)) == EINVAL
    s, flagged = ssm_shape(), ssm_shape(dtype=0x101)
    assert lib.dn_ssm_bwd_workspace(ctypes.byref(flagged)) == lib.dn_ssm_bwd_workspace(ctypes.byref(s)) > 0
    assert ssm_bwd(lib, flagged, ws=None) == ENOWS
    assert lib.dn_ssm_step(2, 4, 2, 64, 64, 0x101, P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, None, P(FAKE),
                           P(FAKE), None) == EINVAL
    assert lib.dn_conv_silu_step(2, 2, 16, 4, 0x101, P(FAKE), P(FAKE), None, P(FAKE), P(FAKE), None) == EINVAL
    assert lib.dn_conv_silu(2, 8, 2, 16, 4, 2, 0x102, P(FAKE), P(FAKE), None, None, None, P(FAKE), None, None) == EINVAL
    assert lib.dn_conv_silu_bwd(2, 8, 2, 16, 4, 2, 0x101, P(FAKE), P(FAKE), None, None, None, P(FAKE), None, P(FAKE),
                                P(FAKE), None, None, None, 0, None) == ENOWS
    assert lib.dn_gated_norm(8, 64, 1, 0x101, P(FAKE), P(FAKE), P(FAKE), 1e-5, 0, P(FAKE), None) == EINVAL
