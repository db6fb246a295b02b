"""Which sizes the state space mixer's calls take: launches that do not take
place refuse nothing.  The checks need no GPU: what is accepted goes on to the
workspace's check, which fails here."""
import ctypes

import pytest
import torch

import chunkwise_delta_rule_wy_amd as dn
from test_mixer_ref import ENOWS, EUNSUPPORTED, ssm_bwd, ssm_fwd, ssm_shape


@pytest.fixture(scope="module")
def lib():
    return dn.load_library()


def test_scan_limits_are_those_of_the_launches(lib):
    # 2^23 chunks of two heads: forwards no launch counts chunks, backwards one does (2^24 of them are too many)
    long = ssm_shape(B=1, n_seqs=1, T=1 << 29, H=2, G=1)
    assert ssm_fwd(lib, long, ws=None) == ENOWS
    half = ssm_shape(B=1, n_seqs=1, T=1 << 28, H=4, G=1)
    assert ssm_bwd(lib, half, ws=None) == ENOWS
    longer = ssm_shape(B=1, n_seqs=1, T=1 << 30, H=2, G=1)
    assert ssm_fwd(lib, longer, ws=None) == ENOWS and ssm_bwd(lib, longer, ws=None) == EUNSUPPORTED
    # 2^20 states of 128 x 128: only sequences that are cut are joined
    many = ssm_shape(B=1 << 20, n_seqs=1 << 20, T=1, H=1, G=1, Dk=128, Dv=128)
    assert ssm_bwd(lib, many, ws=None) == ENOWS


def test_scan_sizes_do_not_wrap(lib):
    top = (1 << 31) - 1
    for kw in (dict(H=1 << 17, G=1 << 17), dict(H=1, G=1), dict(H=1 << 18, G=1)):
        s = ssm_shape(B=top, n_seqs=top, T=top, **kw)
        assert ssm_bwd(lib, s) == EUNSUPPORTED and ssm_fwd(lib, s) == EUNSUPPORTED
    p = ssm_shape(B=1, n_seqs=top, T=top, H=1 << 17, G=1 << 17)
    assert lib.dn_ssm_fwd(ctypes.byref(p), *[0x10000] * 5, None, None, None, 0x10000, 0x10000, None, 0x10000, 1 << 60,
                          None) == EUNSUPPORTED


@pytest.mark.gpu
def test_scan_of_very_many_sequences():
    # one token each, more states than a join would have workgroups for: o = (s q.k + skip) v
    N, dk, dv = 524289, 128, 128
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v = (torch.randn(N, 1, 1, d, generator=g, device="cuda").to(torch.bfloat16) for d in (dk, dk, dv))
    dt, A, skip = torch.randn(N, 1, 1, generator=g, device="cuda"), -torch.ones(1).cuda(), torch.ones(1).cuda()
    o, hT = dn.ssm_fwd(q, k, v, dt, A, None, skip, output_final_state=False)
    assert hT is None
    s = torch.logaddexp(dt.double(), torch.zeros_like(dt, dtype=torch.float64))[..., None]
    terms = (q.double() * k.double())
    want = (s * terms.sum(-1, keepdim=True) + 1) * v.double()
    # P is rounded to bf16 once (half a step of the sum, its fp32 sum over dk before it), and o once
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 * (s * terms.sum(-1, keepdim=True)).abs() * (1 + 2.0 ** -6)
                                      + 2.0 ** -24 * (dk + 16) * (s * terms.abs().sum(-1, keepdim=True) + 1)) * v.double().abs()
    assert ((o.double() - want).abs() <= bound).all()


def conv_bwd(lib, n_seqs, ds0, W=4, H=1, D=256, T=8, wsb=0):
    F = 0x10000
    return lib.dn_conv_silu_bwd(1, T, H, D, W, n_seqs, 1, F, F, None, None, F, F, None, F, F, None, ds0, F, wsb, None)


def test_convolution_takes_any_number_of_sequences(lib):
    # the backward pass as well as the forward one, with or without gradients of the states
    for n in (300000, 1 << 30):
        for ds0 in (None, 0x10000):
            assert conv_bwd(lib, n, ds0) == ENOWS
            assert conv_bwd(lib, n, ds0, W=1) == ENOWS


@pytest.mark.gpu
@pytest.mark.parametrize("H,D,N", [(2, 128, 270001), (1, 8, 1048600)])
def test_convolution_of_very_many_sequences(H, D, N):
    # nearly all without tokens, which pass their state's gradient on; a few with some
    lens = torch.zeros(N, dtype=torch.int64)
    at = [0, 5, N // 2, N - 2, N - 1]
    lens[at] = torch.tensor([3, 1, 40, 2, 9])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
    T, W = int(lens.sum()), 2
    g = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, dy, s0, dsT = r(1, T, H, D), r(1, T, H, D), r(N, W - 1, H, D), r(N, W - 1, H, D)
    w, b = r(H, D, W).float(), r(H, D).float()
    y, sT = dn.conv_silu(x, w, b, s0, cu)
    gr = dn.conv_silu_bwd(x, w, b, s0, dy, dsT, cu)
    empty = (lens == 0).cuda()
    assert torch.equal(sT[empty], s0[empty]) and torch.equal(gr["ds0"][empty], dsT[empty])
    few = torch.cat([torch.zeros(1, dtype=torch.int64), lens[at].cumsum(0)]).to(torch.int32).cuda()
    y0, sT0 = dn.conv_silu(x, w, b, s0[at], few)
    g0 = dn.conv_silu_bwd(x, w, b, s0[at], dy, dsT[at], few)
    assert torch.equal(y, y0) and torch.equal(sT[at], sT0) and torch.equal(gr["ds0"][at], g0["ds0"])
    assert all(torch.equal(gr[n], g0[n]) for n in ("dx", "dw", "dbias"))


@pytest.mark.gpu
def test_convolution_of_very_many_channels():
    # 2^28 sums of weights' gradients and more; the last channels against the same by themselves
    H, D, W, T, last = 128, (1 << 20) + 8, 1, 3, 16
    g = torch.Generator("cuda").manual_seed(6)
    x, dy = (torch.randn(1, T, H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w, b = (torch.randn(H, D, *s, generator=g, device="cuda") for s in ((W,), ()))
    assert H * D * (W + 1) >= 1 << 28
    gr = dn.conv_silu_bwd(x, w, b, None, dy)
    cut = lambda t: t[..., -1:, -last:].contiguous()  # noqa: E731
    g0 = dn.conv_silu_bwd(cut(x), w[-1:, -last:].contiguous(), cut(b), None, cut(dy))
    assert torch.equal(cut(gr["dx"]), g0["dx"])
    assert torch.equal(gr["dw"][-1:, -last:], g0["dw"]) and torch.equal(cut(gr["dbias"]), g0["dbias"])
    first = dn.conv_silu_bwd(x[:, :, :1, :64].contiguous(), w[:1, :64].contiguous(), b[:1, :64].contiguous(), None,
                             dy[:, :, :1, :64].contiguous())
    assert torch.equal(gr["dw"][:1, :64], first["dw"])


def norm_bwd(lib, R, rows=None, ws=None):
    F = 0x10000
    return lib.dn_gated_norm_bwd(rows or R, 8, R, 1, F, F, F, 1e-5, 0, F, F, F, F, ws, 0, None)


def test_norm_takes_any_number_of_heads(lib):
    assert norm_bwd(lib, 65536) == ENOWS and norm_bwd(lib, (1 << 24) - 1) == ENOWS
    assert norm_bwd(lib, 1 << 24) == EUNSUPPORTED  # 2^32 threads


@pytest.mark.gpu
@pytest.mark.parametrize("first", [False, True])
def test_norm_of_very_many_heads(first):
    # three heads alone get the same gradients as among 70001
    R, D, n = 70001, 24, 3
    g = torch.Generator("cuda").manual_seed(7)
    x, z, dy = (torch.randn(n, R, D, generator=g, device="cuda") for _ in range(3))
    w = torch.randn(R, D, generator=g, device="cuda")
    got = dn.gated_norm_bwd(x, z, w, dy, gate_first=first)
    for at in ([0, 1, 2], [65534, 65535, 65536], [R - 3, R - 2, R - 1]):
        cut = lambda t: t[:, at].contiguous()  # noqa: E731
        want = dn.gated_norm_bwd(cut(x), cut(z), w[at], cut(dy), gate_first=first)
        assert torch.equal(cut(got[0]), want[0]) and torch.equal(cut(got[1]), want[1])
        # three terms, added in some order
        size = (dy.abs() * dn.gated_norm(x, z, w, gate_first=first).abs() / w.abs()).sum(0)[at]
        assert ((got[2][at] - want[2]).abs() <= 8 * 2.0 ** -24 * size).all()
