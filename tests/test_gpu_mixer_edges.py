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
