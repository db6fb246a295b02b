// C ABI of the selective state space scan: argument validation, the plan of
// segments, workspace layout and launches.  Like the other entry points these
// validate on the host, enqueue nothing on error, and never allocate, free or
// synchronise.
#include "dn.h"
#include "dn_internal.h"
#include "dn_ssm.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

dn_status check_dims(int32_t H, int32_t G, int32_t Dk, int32_t Dv, int32_t dtype) {
  if (H <= 0 || G <= 0 || Dk <= 0 || Dv <= 0 || H % G != 0) return DN_EINVAL;
  if (dtype != DN_F32 && dtype != DN_BF16) return DN_EINVAL;
  if ((Dk != 64 && Dk != 128) || Dv % 64 != 0 || Dv > 1024) return DN_EUNSUPPORTED;
  return DN_OK;
}

dn_status check_shape(const dn_ssm_shape *s, bool packed) {
  if (!s || s->B <= 0 || s->T < 0 || s->n_seqs <= 0) return DN_EINVAL;
  const dn_status st = check_dims(s->H, s->G, s->Dk, s->Dv, s->dtype & ~DN_ZERO_TAIL);
  if (st != DN_OK) return st;
  if (packed ? s->B != 1 : s->n_seqs != s->B) return DN_EINVAL;
  if ((s->dtype & ~DN_ZERO_TAIL) != DN_BF16) return DN_EUNSUPPORTED;  // the chunk kernels are bf16
  // the kernels address a chunk's rows with 32-bit byte offsets
  if ((int64_t)128 * s->H * s->Dv > INT32_MAX || (int64_t)128 * s->G * s->Dk > INT32_MAX) return DN_EUNSUPPORTED;
  return DN_OK;
}

// Two column tiles share a workgroup where Dv has them, else two heads that
// share their keys (SsmPair): keys and queries then pass through LDS once for
// both.  That gains where workgroups fill the device (whole calls, single tiles
// in brackets: 4 x 4096 tokens, 32 heads of 128 x 64, both passes, 519 us [543];
// 16384 tokens, 16 heads of 128 x 128, 118 [127]; 65536 packed ones, 32 heads, 802
// [903]; 2048 tokens, 512 heads, 266 [312]) and loses where few of them walk an
// uncut chain of chunks (2048 tokens, 4 to 128 heads of 128 x 128, 133 to 142 us
// [104 to 108]; 128 x 64, both passes, 4 to 64 heads, 260 to 297 [200 to 236]; 1357
// ragged ones 61 [58]): the rule does not tell these apart.
int pair_of(const dn_ssm_shape *s) {
  if (s->Dv % 128 == 0) return dn::SSM_TILES;
  return (s->H / s->G) % 2 == 0 ? dn::SSM_HEADS : dn::SSM_SINGLE;
}

// Segments (whole chunks of one sequence) and their tables.
//
// A segment costs a sweep over its tokens and passes over its state, so that
// sequences are cut only where they would leave compute units idle.
// Up to UNCUT chunks nothing is cut: the chunks' chain is then no longer than
// the three passes that cutting needs (1357 tokens in 9 sequences, 6 heads,
// 64 x 128, forwards and backwards: 65 us, cut into segments of 4 chunks 80 us).
// Fixed length: no cuts from FULL_WGS workgroups on, else about FIXED_WGS, two
// for each of the 256 CUs, and not below four chunks a segment (16384 tokens,
// 16 heads, 128 x 128: 125 us, with 384 workgroups 142 us, 1024: 149 us).
// Packed: the lengths are not known on the host, and one long sequence among
// short ones would set the pass's time, so that longer packs are always cut, so
// finely that the workgroups' rounds come out even (65536 tokens, 32 heads,
// 128 x 128: 833 us with PACKED_WGS 2048, 906 us with 1024, 882 us with 4096).
constexpr int64_t UNCUT = 32, FULL_WGS = 384, FIXED_WGS = 512, PACKED_WGS = 2048;

struct Plan {
  int split, NS, segc, NC;
  int64_t nseg, nchunks;
};

Plan plan_of(const dn_ssm_shape *s, bool packed, bool backward) {
  Plan p = {};
  const int64_t tiles = (int64_t)s->H * (s->Dv / 64) / (pair_of(s) == dn::SSM_SINGLE ? 1 : 2), chunks = ((int64_t)s->T + 63) / 64;
  p.NC = (int)chunks;
  if (packed) {
    const int64_t want = (chunks * tiles + PACKED_WGS - 1) / PACKED_WGS;
    p.segc = (int)(want < 4 ? 4 : want > 1 << 20 ? 1 << 20 : want);
    if (chunks <= UNCUT) p.segc = (int)(chunks < 1 ? 1 : chunks);
    p.split = p.segc < chunks;
    p.nseg = (p.split ? (int64_t)s->T / (64 * (int64_t)p.segc) : 0) + s->n_seqs;
    p.nchunks = (int64_t)s->T / 64 + s->n_seqs;
    return p;
  }
  const int64_t streams = tiles * s->n_seqs * (backward ? 2 : 1);  // the backward pass sweeps both ways at once
  int64_t ns = streams >= FULL_WGS || chunks <= UNCUT ? 1 : (FIXED_WGS + streams - 1) / streams;
  if (ns > chunks / 4) ns = chunks / 4;
  if (ns < 1) ns = 1;
  p.segc = (int)((chunks + ns - 1) / ns);
  if (p.segc < 1) p.segc = 1;
  p.NS = chunks > 0 ? (int)((chunks + p.segc - 1) / p.segc) : 1;
  p.split = p.NS > 1;
  p.nseg = (int64_t)p.NS * s->n_seqs;
  p.nchunks = chunks * s->n_seqs;
  return p;
}

// Sets of a group's heads for the gradient kernel: one workgroup per CU where
// the heads give as many, since every set costs a start and a share of fp32
// partial sums (4 x 4096 tokens, 32 heads: 198 us with one set, 234 us with
// four, their sums included).
void sets_of(const dn_ssm_shape *s, const Plan &pl, int &sets, int &heads) {
  const int64_t R = s->H / s->G, wgs = (pl.nchunks < 256 ? pl.nchunks : 256) * s->G;  // 256 fill it
  int64_t n = wgs > 0 ? (256 + wgs - 1) / wgs : 1;
  if (n > R) n = R;
  heads = (int)((R + n - 1) / n);
  sets = (int)((R + heads - 1) / heads);
}

struct Layout {
  size_t tables, decay, seg[2], states, dstates, part, dq_part, dk_part, total;
};

Layout layout_of(const dn_ssm_shape *s, const Plan &pl, bool packed, bool backward) {
  Layout L = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align256(bytes);
    return x;
  };
  const size_t st = (size_t)s->H * s->Dk * s->Dv * 4;
  if (packed)
    L.tables = take(4 * ((pl.split ? (size_t)s->n_seqs + 1 + pl.nseg : 0) +
                         (backward ? (size_t)s->n_seqs + 1 + pl.nchunks : 0)));
  if (pl.split) {
    L.decay = take(8 * (size_t)pl.nseg * s->H);
    for (int i = 0; i < (backward ? 2 : 1); ++i) L.seg[i] = take((size_t)pl.nseg * st);
  }
  if (backward) {
    L.states = take((size_t)pl.nchunks * st);
    L.dstates = take((size_t)pl.nchunks * st);
    L.part = take(24 * (size_t)pl.nchunks * s->H);
    int sets, heads;
    sets_of(s, pl, sets, heads);
    if (sets > 1) {
      const size_t n = 4 * (size_t)sets * s->B * s->T * s->G * s->Dk;
      L.dq_part = take(n);
      L.dk_part = take(n);
    }
  }
  L.total = at;
  return L;
}

// The queries cannot see cu_seqlens: with one batch row the input may be
// packed, and the answer covers both plans.
size_t workspace(const dn_ssm_shape *s, bool backward) {
  if (!s || s->B <= 0 || s->T < 0 || s->n_seqs <= 0) return 0;
  if (check_dims(s->H, s->G, s->Dk, s->Dv, s->dtype & ~DN_ZERO_TAIL) != DN_OK) return 0;
  size_t n = 0;
  if (s->n_seqs == s->B) n = layout_of(s, plan_of(s, false, backward), false, backward).total;
  if (s->B == 1) {
    const size_t m = layout_of(s, plan_of(s, true, backward), true, backward).total;
    if (m > n) n = m;
  }
  return n;
}

// Checks the grids' sizes and the workspace, fills the parameters and builds
// the packed tables.
dn_status setup(const dn_ssm_shape *s, const int32_t *cu, bool backward, void *ws, size_t ws_bytes, dn::SsmParams &p,
                hipStream_t stream) {
  const bool packed = cu != nullptr;
  const Plan pl = plan_of(s, packed, backward);
  // a grid has fewer than 2^32 threads, in workgroups of up to 512: segments, the
  // join's states, and the gradient kernel's chunks
  const int64_t top = UINT32_MAX / 512;
  if (pl.nseg * s->H * (s->Dv / 64) > top) return DN_EUNSUPPORTED;
  if (pl.split && (int64_t)s->n_seqs * s->H * (s->Dk * s->Dv / 1024) > top) return DN_EUNSUPPORTED;
  sets_of(s, pl, p.sets, p.set_heads);
  if (backward && (pl.nchunks > top || pl.nchunks * s->G * p.sets > top)) return DN_EUNSUPPORTED;
  const Layout L = layout_of(s, pl, packed, backward);
  if (L.total > 0 && (ws_bytes < L.total || !ws || !aligned16(ws))) return DN_ENOWS;
  char *base = static_cast<char *>(ws);
  p.cu = cu;
  p.zero_tail = packed && (s->dtype & DN_ZERO_TAIL) != 0;
  p.rows = (int64_t)s->B * s->T;
  p.T = s->T;
  p.H = s->H;
  p.G = s->G;
  p.DV = s->Dv;
  p.N = s->n_seqs;
  p.ntiles = s->Dv / 64;
  p.pair = pair_of(s);
  p.split = pl.split;
  p.NS = pl.NS;
  p.segc = pl.segc;
  p.NC = pl.NC;
  p.nseg = (int)pl.nseg;
  p.nchunks = (int)pl.nchunks;
  if (pl.split) {
    p.seg_decay = reinterpret_cast<double *>(base + L.decay);
    for (int i = 0; i < (backward ? 2 : 1); ++i) p.seg_state[i] = reinterpret_cast<float *>(base + L.seg[i]);
  }
  if (backward) {
    p.states = reinterpret_cast<float *>(base + L.states);
    p.dstates = reinterpret_cast<float *>(base + L.dstates);
    p.par_part = reinterpret_cast<double *>(base + L.part);
    if (p.sets > 1) {
      p.dq_part = reinterpret_cast<float *>(base + L.dq_part);
      p.dk_part = reinterpret_cast<float *>(base + L.dk_part);
    }
  }
  if (packed) {
    int32_t *t = reinterpret_cast<int32_t *>(base + L.tables);
    if (pl.split) {
      p.seg_base = t;
      p.seg_seq = t + s->n_seqs + 1;
      if (dn::launch_chunk_table(cu, s->n_seqs, t, t + s->n_seqs + 1, p.nseg, 64 * p.segc, stream) != hipSuccess)
        return DN_EHIP;
      t += s->n_seqs + 1 + pl.nseg;
    }
    if (backward) {
      p.chunk_base = t;
      p.chunk_seq = t + s->n_seqs + 1;
      if (dn::launch_chunk_table(cu, s->n_seqs, t, t + s->n_seqs + 1, p.nchunks, 64, stream) != hipSuccess)
        return DN_EHIP;
    }
  }
  return DN_OK;
}

bool all16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (!aligned16(p)) return false;
  return true;
}

}  // namespace

extern "C" size_t dn_ssm_fwd_workspace(const dn_ssm_shape *s) { return workspace(s, false); }
extern "C" size_t dn_ssm_bwd_workspace(const dn_ssm_shape *s) { return workspace(s, true); }

extern "C" dn_status dn_ssm_fwd(const dn_ssm_shape *s, const void *q, const void *k, const void *v, const float *dt,
                                const float *A, const float *dt_bias, const float *skip, const float *h0,
                                const int32_t *cu_seqlens, void *o, float *hT, void *workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  dn_status st = check_shape(s, cu_seqlens != nullptr);
  if (st != DN_OK) return st;
  if (!A || !all16({h0, hT})) return DN_EINVAL;
  if (s->T > 0 && (!q || !k || !v || !dt || !o || !all16({q, k, v, o}))) return DN_EINVAL;
  dn::SsmParams p = {};
  p.q = static_cast<const bf16 *>(q);
  p.k = static_cast<const bf16 *>(k);
  p.v = static_cast<const bf16 *>(v);
  p.dt = dt;
  p.A = A;
  p.bias = dt_bias;
  p.skip = skip;
  p.h0 = h0;
  p.o = static_cast<bf16 *>(o);
  p.hT = hT;
  st = setup(s, cu_seqlens, false, workspace, workspace_bytes, p, stream);
  if (st != DN_OK) return st;
  if (p.split) {
    if (dn::launch_ssm_sweep(p, s->Dk, false, false, stream) != hipSuccess) return DN_EHIP;
    if (dn::launch_ssm_join(p, s->Dk, false, stream) != hipSuccess) return DN_EHIP;
  }
  return dn::launch_ssm_fwd(p, s->Dk, stream) == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" dn_status dn_ssm_bwd(const dn_ssm_shape *s, const void *q, const void *k, const void *v, const float *dt,
                                const float *A, const float *dt_bias, const float *skip, const float *h0,
                                const int32_t *cu_seqlens, const void *dO, const float *dhT, void *dq, void *dk,
                                void *dv, float *ddt, float *dA, float *ddt_bias, float *dskip, float *dh0,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
  dn_status st = check_shape(s, cu_seqlens != nullptr);
  if (st != DN_OK) return st;
  if (!A || !dA || !all16({h0, dhT, dh0})) return DN_EINVAL;
  if (s->T > 0 && (!q || !k || !v || !dt || !dO || !dq || !dk || !dv || !ddt || !all16({q, k, v, dO, dq, dk, dv})))
    return DN_EINVAL;
  dn::SsmParams p = {};
  p.q = static_cast<const bf16 *>(q);
  p.k = static_cast<const bf16 *>(k);
  p.v = static_cast<const bf16 *>(v);
  p.dO = static_cast<const bf16 *>(dO);
  p.dt = dt;
  p.A = A;
  p.bias = dt_bias;
  p.skip = skip;
  p.h0 = h0;
  p.dhT = dhT;
  p.dq = static_cast<bf16 *>(dq);
  p.dk = static_cast<bf16 *>(dk);
  p.dv = static_cast<bf16 *>(dv);
  p.ddt = ddt;
  p.dA = dA;
  p.ddt_bias = ddt_bias;
  p.dskip = dskip;
  p.dh0 = dh0;
  st = setup(s, cu_seqlens, true, workspace, workspace_bytes, p, stream);
  if (st != DN_OK) return st;
  if (p.split) {
    if (dn::launch_ssm_sweep(p, s->Dk, false, true, stream) != hipSuccess) return DN_EHIP;
    if (dn::launch_ssm_join(p, s->Dk, true, stream) != hipSuccess) return DN_EHIP;
  }
  if (dn::launch_ssm_sweep(p, s->Dk, true, true, stream) != hipSuccess) return DN_EHIP;
  return dn::launch_ssm_grad(p, s->Dk, stream) == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" dn_status dn_ssm_step(int32_t B, int32_t H, int32_t G, int32_t Dk, int32_t Dv, int32_t dtype, const void *q,
                                 const void *k, const void *v, const float *dt, const float *A, const float *dt_bias,
                                 const float *skip, float *state, void *o, hipStream_t stream) {
  if (B <= 0) return DN_EINVAL;
  const dn_status st = check_dims(H, G, Dk, Dv, dtype);
  if (st != DN_OK) return st;
  if (!q || !k || !v || !dt || !A || !state || !o || !all16({q, k, v, state, o})) return DN_EINVAL;
  if ((int64_t)B * H * (Dv / 64) > UINT32_MAX / 512) return DN_EUNSUPPORTED;
  dn::SsmStepParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.dt = dt;
  p.A = A;
  p.bias = dt_bias;
  p.skip = skip;
  p.state = state;
  p.o = o;
  p.B = B;
  p.H = H;
  p.G = G;
  p.DV = Dv;
  return dn::launch_ssm_step(p, dtype, Dk, stream) == hipSuccess ? DN_OK : DN_EHIP;
}
