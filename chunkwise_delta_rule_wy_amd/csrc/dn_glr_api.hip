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
// where sequences and channels give few workgroups: fewer than FULL_FWD, or up to half of
// WANT backwards, whose maps need one tensor less (4096 rows in bf16, forwards and
// backwards in us, uncut [cut]: 104 workgroups 90 + 159 [125 + 135]; 128 of them 99 + 161 [105 +
// 136]; 160 104 + 183 [179 + 212]; 64 of 16384 packed rows 398 + 715 [203 + 264]), and then up to
// about WANT, one for each CU (those packed rows with 512: 223 + 281, with 1024: 229 +
// 293, with 128: 366 + 474; 16384 rows of 2048 channels with 256: 103 + 131, with 512:
// 110 + 141).
constexpr int64_t FLAT = 512, FULL_FWD = 100, WANT = 256, FULL_BWD = WANT / 2 + 1;

struct Plan {
  bool flat, cut;
  int64_t NS, segt, nseg;
  int64_t states;  // the same for both directions
};

Plan plan_of(int64_t B, int64_t T, int64_t C, bool packed, bool backward) {
  Plan p = {};
  const int64_t groups = (C + dn::GLR_CH - 1) / dn::GLR_CH;
  p.flat = packed || T < FLAT;
  const int64_t rows = p.flat ? B * T : T, tiles = (rows + dn::GLR_TILE - 1) / dn::GLR_TILE;
  const int64_t streams = groups * (p.flat ? 1 : B);
  int64_t ns = streams >= (backward ? FULL_BWD : FULL_FWD) ? 1 : (WANT + streams - 1) / streams;
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

// Forwards by the plan f, backwards by b; `states`: the backward pass is given them, and
// does not run forwards first.
Layout layout_of(const Plan &f, const Plan &b, int64_t C, bool backward, bool states) {
  Layout L = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align256(bytes);
    return x;
  };
  auto maps = [&](const Plan &p) { return p.cut ? 8 * (size_t)p.nseg * C : 0; };
  L.sum_f = take(backward && states ? 0 : maps(f));
  if (backward) {
    L.sum_r = take(maps(b));
    L.part = take(12 * (size_t)b.nseg * C);
    if (!states) L.states = take(4 * (size_t)b.states * C);
  }
  L.total = at;
  return L;
}

// The queries cannot see cu_seqlens: with one batch row the input may be packed.
template <typename F>
size_t most(int32_t B, int32_t T, int32_t H, int32_t D, F of) {
  if (B <= 0 || T < 0 || H <= 0 || D <= 0 || (int64_t)H * D > MAX_C || (int64_t)B * T > INT32_MAX) return 0;
  const int64_t C = (int64_t)H * D;
  size_t n = of(plan_of(B, T, C, false, false), plan_of(B, T, C, false, true));
  if (B == 1) {
    const size_t m = of(plan_of(B, T, C, true, false), plan_of(B, T, C, true, true));
    if (m > n) n = m;
  }
  return n;
}

void set_plan(dn::GlrParams &p, const Plan &pl) {
  p.flat = pl.flat;
  p.NS = (int)pl.NS;
  p.segt = (int)pl.segt;
  p.nseg = (int)pl.nseg;
  p.cut = pl.cut;
}

dn_status setup(dn::GlrParams &p, int32_t B, int32_t T, int32_t H, int32_t D, int32_t n_seqs, int32_t dtype,
                const int32_t *cu, float power, bool backward, void *ws, size_t ws_bytes) {
  p.C = H * D;
  const Plan f = plan_of(B, T, p.C, cu != nullptr, false), b = plan_of(B, T, p.C, cu != nullptr, true);
  p.groups = (p.C + dn::GLR_CH - 1) / dn::GLR_CH;
  // a grid has fewer than 2^32 threads
  if ((f.nseg > b.nseg ? f.nseg : b.nseg) * p.groups > UINT32_MAX / dn::GLR_THREADS) return DN_EUNSUPPORTED;
  const Layout L = layout_of(f, b, p.C, backward, p.states != nullptr);
  if (L.total > 0 && (!ws || !all16({ws}) || ws_bytes < L.total)) return DN_ENOWS;
  char *base = static_cast<char *>(ws);
  p.cu = cu;
  p.rows = (int64_t)B * T;
  p.T = T;
  p.N = n_seqs;
  set_plan(p, backward ? b : f);
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
  return most(B, T, H, D, [](const Plan &f, const Plan &) { return (size_t)f.states; });
}

extern "C" size_t dn_glr_fwd_workspace(int32_t B, int32_t T, int32_t H, int32_t D) {
  return most(B, T, H, D, [=](const Plan &f, const Plan &b) { return layout_of(f, b, (int64_t)H * D, false, true).total; });
}

extern "C" size_t dn_glr_bwd_workspace(int32_t B, int32_t T, int32_t H, int32_t D, int32_t with_states) {
  return most(B, T, H, D, [=](const Plan &f, const Plan &b) { return layout_of(f, b, (int64_t)H * D, true, with_states != 0).total; });
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
  // without kept states a forward pass, cut as that is, writes the same ones, and nothing else
  if (!states) {
    dn::GlrParams f = p;
    set_plan(f, plan_of(B, T, p.C, cu_seqlens != nullptr, false));
    st = forward(f, e, stream);
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
