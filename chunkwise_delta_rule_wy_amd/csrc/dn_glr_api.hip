// C ABI of the gated linear recurrence: argument validation, the plan of
// segments, workspace layout and launches.
#include "dn.h"
#include "dn_glr.h"

namespace {

constexpr int64_t MAX_C = 1 << 23;  // a tile's rows are addressed with 32-bit element offsets

bool all16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return true;
}
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

dn_status check(int32_t B, int32_t T, int32_t H, int32_t D, int32_t n_seqs, int32_t dtype, bool packed, float power) {
  const int32_t e = dtype & ~DN_ZERO_TAIL;
  if (B <= 0 || T < 0 || H <= 0 || D <= 0 || n_seqs <= 0 || !(power > 0.f && power <= 3.4e38f)) return DN_EINVAL;
  if (e != DN_F32 && e != DN_BF16) return DN_EINVAL;
  if (packed ? B != 1 : n_seqs != B) return DN_EINVAL;
  if (D % 8 != 0 || (int64_t)H * D > MAX_C || (int64_t)B * T > INT32_MAX) return DN_EUNSUPPORTED;
  return DN_OK;
}

// Segments.  Sequences of FLAT rows and more are cut by themselves, packed and
// shorter ones lie in one run of rows that is cut evenly, whatever their lengths.
// Cutting reads the inputs twice (the segments' maps first), so that it pays only
// where sequences and channels give fewer than FULL workgroups (forwards and backwards
// in us, uncut [cut]: 128 workgroups of 4 x 4096 rows in fp32, 143 + 235 [199 + 252]; 64
// of 16384 packed rows, 419 + 695 [243 + 278]), and then up to about WANT, one for each
// CU (the packed rows with 512: 238 + 286, with 1024: 243 + 302, with 128: 401 + 471; 16384
// rows of 2048 channels with 256: 112 + 143, with 512: 116 + 150).
constexpr int64_t FLAT = 512, FULL = 100, WANT = 256;

struct Plan {
  bool flat, cut;
  int64_t NS, segt, nseg, states;
};

Plan plan_of(int64_t B, int64_t T, int64_t C, bool packed) {
  Plan p = {};
  const int64_t groups = (C + dn::GLR_CH - 1) / dn::GLR_CH;
  p.flat = packed || T < FLAT;
  const int64_t rows = p.flat ? B * T : T, tiles = (rows + dn::GLR_TILE - 1) / dn::GLR_TILE;
  const int64_t streams = groups * (p.flat ? 1 : B);
  int64_t ns = streams >= FULL ? 1 : (WANT + streams - 1) / streams;
  if (ns > tiles) ns = tiles;
  if (ns < 1) ns = 1;
  p.segt = (tiles + ns - 1) / ns;
  if (p.segt < 1) p.segt = 1;
  p.NS = tiles > 0 ? (tiles + p.segt - 1) / p.segt : 1;
  p.nseg = p.NS * (p.flat ? 1 : B);
  p.cut = p.NS > 1;
  p.states = (rows + dn::GLR_STATE - 1) / dn::GLR_STATE * (p.flat ? 1 : B);
  return p;
}

struct Layout {
  size_t sum_f, sum_r, part, states, total;
};

Layout layout_of(const Plan &p, int64_t C, bool backward, bool states) {
  Layout L = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align256(bytes);
    return x;
  };
  const size_t maps = p.cut ? 8 * (size_t)p.nseg * C : 0;
  L.sum_f = take(backward && states ? 0 : maps);
  if (backward) {
    L.sum_r = take(maps);
    L.part = take(12 * (size_t)p.nseg * C);
    if (!states) L.states = take(4 * (size_t)p.states * C);
  }
  L.total = at;
  return L;
}

// The queries cannot see cu_seqlens: with one batch row the input may be packed.
template <typename F>
size_t most(int32_t B, int32_t T, int32_t H, int32_t D, F of) {
  if (B <= 0 || T < 0 || H <= 0 || D <= 0 || (int64_t)H * D > MAX_C || (int64_t)B * T > INT32_MAX) return 0;
  size_t n = of(plan_of(B, T, (int64_t)H * D, false));
  if (B == 1) {
    const size_t m = of(plan_of(B, T, (int64_t)H * D, true));
    if (m > n) n = m;
  }
  return n;
}

dn_status setup(dn::GlrParams &p, int32_t B, int32_t T, int32_t H, int32_t D, int32_t n_seqs, int32_t dtype,
                const int32_t *cu, float power, bool backward, void *ws, size_t ws_bytes) {
  p.C = H * D;
  const Plan pl = plan_of(B, T, p.C, cu != nullptr);
  p.groups = (p.C + dn::GLR_CH - 1) / dn::GLR_CH;
  // a grid has fewer than 2^32 threads
  if (pl.nseg * p.groups > UINT32_MAX / dn::GLR_THREADS) return DN_EUNSUPPORTED;
  const Layout L = layout_of(pl, p.C, backward, p.states != nullptr);
  if (L.total > 0 && (!ws || !all16({ws}) || ws_bytes < L.total)) return DN_ENOWS;
  char *base = static_cast<char *>(ws);
  p.cu = cu;
  p.rows = (int64_t)B * T;
  p.T = T;
  p.N = n_seqs;
  p.flat = pl.flat;
  p.NS = (int)pl.NS;
  p.segt = (int)pl.segt;
  p.nseg = (int)pl.nseg;
  p.cut = pl.cut;
  p.zero_tail = cu && (dtype & DN_ZERO_TAIL);
  p.power = power;
  p.sum_f = reinterpret_cast<float *>(base + L.sum_f);
  if (backward) {
    p.sum_r = reinterpret_cast<float *>(base + L.sum_r);
    p.part = reinterpret_cast<float *>(base + L.part);
    if (!p.states) p.states = reinterpret_cast<float *>(base + L.states);
  }
  return DN_OK;
}

dn_status forward(const dn::GlrParams &p, int dtype, hipStream_t stream) {
  if (p.cut && dn::launch_glr_sum(p, dtype, false, stream) != hipSuccess) return DN_EHIP;
  return dn::launch_glr_fwd(p, dtype, stream) == hipSuccess ? DN_OK : DN_EHIP;
}

}  // namespace

extern "C" size_t dn_glr_states(int32_t B, int32_t T, int32_t H, int32_t D) {
  return most(B, T, H, D, [](const Plan &p) { return (size_t)p.states; });
}

extern "C" size_t dn_glr_fwd_workspace(int32_t B, int32_t T, int32_t H, int32_t D) {
  return most(B, T, H, D, [=](const Plan &p) { return layout_of(p, (int64_t)H * D, false, true).total; });
}

extern "C" size_t dn_glr_bwd_workspace(int32_t B, int32_t T, int32_t H, int32_t D, int32_t with_states) {
  return most(B, T, H, D, [=](const Plan &p) { return layout_of(p, (int64_t)H * D, true, with_states != 0).total; });
}

extern "C" dn_status dn_glr_fwd(int32_t B, int32_t T, int32_t H, int32_t D, int32_t n_seqs, int32_t dtype, const void *x,
                                const void *r, const void *i, const float *lam, const float *br, const float *bi,
                                float power, const float *h0, const int32_t *cu_seqlens, void *y, float *hT, float *states,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
  dn_status st = check(B, T, H, D, n_seqs, dtype, cu_seqlens != nullptr, power);
  if (st != DN_OK) return st;
  if (!lam || !all16({h0, hT, states})) return DN_EINVAL;
  if (T > 0 && (!x || !r || !i || !y || !all16({x, r, i, y}))) return DN_EINVAL;
  dn::GlrParams p = {};
  p.x = x;
  p.r = r;
  p.i = i;
  p.lam = lam;
  p.br = br;
  p.bi = bi;
  p.h0 = h0;
  p.y = y;
  p.hT = hT;
  p.states = states;
  st = setup(p, B, T, H, D, n_seqs, dtype, cu_seqlens, power, false, workspace, workspace_bytes);
  return st != DN_OK ? st : forward(p, dtype & ~DN_ZERO_TAIL, stream);
}

extern "C" dn_status dn_glr_bwd(int32_t B, int32_t T, int32_t H, int32_t D, int32_t n_seqs, int32_t dtype, const void *x,
                                const void *r, const void *i, const float *lam, const float *br, const float *bi,
                                float power, const float *h0, const int32_t *cu_seqlens, const float *states,
                                const void *dy, const float *dhT, void *dx, void *dr, void *di, float *dlam, float *dbr,
                                float *dbi, float *dh0, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  dn_status st = check(B, T, H, D, n_seqs, dtype, cu_seqlens != nullptr, power);
  if (st != DN_OK) return st;
  if (!lam || !dlam || !all16({h0, dhT, dh0, states})) return DN_EINVAL;
  if (T > 0 && (!x || !r || !i || !dy || !dx || !dr || !di || !all16({x, r, i, dy, dx, dr, di}))) return DN_EINVAL;
  dn::GlrParams p = {};
  p.x = x;
  p.r = r;
  p.i = i;
  p.dy = dy;
  p.lam = lam;
  p.br = br;
  p.bi = bi;
  p.h0 = h0;
  p.dhT = dhT;
  p.states = const_cast<float *>(states);
  p.dx = dx;
  p.dr = dr;
  p.di = di;
  p.dlam = dlam;
  p.dbr = dbr;
  p.dbi = dbi;
  p.dh0 = dh0;
  st = setup(p, B, T, H, D, n_seqs, dtype, cu_seqlens, power, true, workspace, workspace_bytes);
  if (st != DN_OK) return st;
  const int e = dtype & ~DN_ZERO_TAIL;
  // without kept states a forward pass writes them, and nothing else
  if (!states) {
    st = forward(p, e, stream);
    if (st != DN_OK) return st;
  }
  if (p.cut && dn::launch_glr_sum(p, e, true, stream) != hipSuccess) return DN_EHIP;
  return dn::launch_glr_bwd(p, e, stream) == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" dn_status dn_glr_step(int32_t B, int32_t H, int32_t D, int32_t dtype, const void *x, const void *r,
                                 const void *i, const float *lam, const float *br, const float *bi, float power,
                                 float *state, void *y, hipStream_t stream) {
  const dn_status st = check(B, 1, H, D, B, dtype, false, power);
  if (st != DN_OK) return st;
  if (dtype & DN_ZERO_TAIL) return DN_EINVAL;
  if (!x || !r || !i || !lam || !state || !y || !all16({x, r, i, state, y})) return DN_EINVAL;
  // a grid's rows, and fewer than 2^32 threads
  if (B > 65535 * 4 || ((int64_t)H * D / 4 + 255) / 256 * B > UINT32_MAX / 256) return DN_EUNSUPPORTED;
  dn::GlrStepParams p = {};
  p.x = x;
  p.r = r;
  p.i = i;
  p.lam = lam;
  p.br = br;
  p.bi = bi;
  p.state = state;
  p.y = y;
  p.B = B;
  p.C = H * D;
  p.power = power;
  return dn::launch_glr_step(p, dtype, stream) == hipSuccess ? DN_OK : DN_EHIP;
}
