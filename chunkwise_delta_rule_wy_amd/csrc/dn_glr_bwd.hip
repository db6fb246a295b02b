// Gated linear recurrence, backward pass (dn_glr.h has the mathematics).  A
// workgroup walks through its segment from the last tile to the first.  In a tile
// the states come forwards from the one kept in front of it, and the gradients
// go backwards from the tile behind; both exchanges between the runs share one
// barrier.  The parameters' gradients are summed in registers over the segment,
// in LDS over the runs and by a second kernel over the segments, in a fixed order.
// 4 x 4096 tokens of 4096 channels in bf16 take 195 to 202 us, 4.7 TB/s of four tensors read and
// three written, with vector instructions in 68 % of the cycles.
#include "dn_glr.h"

namespace dn {
namespace {

// Rows of a run: what stays of eight until the gradients passes the registers (4 x 4096
// tokens of 4096 channels in bf16, whole calls: 211 us, with eight 468).
constexpr int BWD_ROWS = 4;

template <typename E, int ROWS, bool FLAT>
__global__ __launch_bounds__(GLR_THREADS) void glr_bwd_kernel(GlrParams p) {
  typedef typename Pair<E>::type P2;
  constexpr int TILE = GLR_RUNS * ROWS;
  static_assert(TILE % GLR_STATE == 0 && GLR_TILE % TILE == 0, "a tile starts with a kept state");
  __shared__ f32x4 fwd_maps[2][GLR_WAVES][GLR_LANES], bwd_maps[2][GLR_WAVES][GLR_LANES];
  __shared__ float sums[3][GLR_RUNS][GLR_CH];
  const int seg = blockIdx.x / p.groups, grp = blockIdx.x % p.groups;
  const int lane = threadIdx.x % GLR_LANES, run = threadIdx.x / GLR_LANES, wave = __builtin_amdgcn_readfirstlane(wave_id());
  // lanes behind the last channels repeat them, stores included
  const int c = min(grp * GLR_CH + 2 * lane, p.C - 2);
  const bool upper = threadIdx.x & 32;
  const GlrSegment s = glr_segment(p, seg);
  const GlrChannel k0 = glr_channel(p.lam, p.br, p.bi, p.power, c), k1 = glr_channel(p.lam, p.br, p.bi, p.power, c + 1);
  // sequences without tokens pass dhT on
  if (p.dh0 && (p.cu || p.T == 0))
    for (int64_t n = (int64_t)seg * GLR_RUNS + run; n < p.N; n += (int64_t)p.nseg * GLR_RUNS)
      if (!p.cu || p.cu[n] == p.cu[n + 1])
        *reinterpret_cast<f32x2 *>(p.dh0 + n * p.C + c) =
            p.dhT ? *reinterpret_cast<const f32x2 *>(p.dhT + n * p.C + c) : (f32x2){0.f, 0.f};
  f32x2 carry = {0.f, 0.f};  // the gradient that reaches the tile from behind
  GlrSeq q;
  const int last = glr_reach<true>(p, s, seg, q);
  if (p.cut) carry = glr_join<true>(p, p.sum_r, seg + 1, last + 1, c, &fwd_maps[0][0][0]);
  f32x2 dlam = {0.f, 0.f}, dbr = {0.f, 0.f}, dbi = {0.f, 0.f};
  const int64_t tiles = (s.row1 - s.row0 + TILE - 1) / TILE;
  P2 x[ROWS], r[ROWS], i[ROWS], dy[ROWS];
  const uint32_t pitch = p.C * (uint32_t)sizeof(E), col = c * (uint32_t)sizeof(E);
  f32x2 kept = {0.f, 0.f};
  // tile t, and the state kept in front of it: a load that is waited for by itself
  // would wait for the others.  No branch: registers that are loaded in one of two
  // ways get copied where these meet, and the copies wait
  const auto load = [&](int64_t t) {
    const int64_t tile = s.row0 + t * TILE;
    uint32_t o[ROWS];
    glr_offsets<ROWS>(o, run * ROWS, (int)min(s.row1 - tile, (int64_t)TILE), pitch, col);
    kept = *reinterpret_cast<const f32x2 *>(p.states + (s.state0 + t * (TILE / GLR_STATE)) * p.C + c);
    glr_load<E>(p.x, tile, o, p.C, x);
    glr_load<E>(p.r, tile, o, p.C, r);
    glr_load<E>(p.i, tile, o, p.C, i);
    glr_load<E>(p.dy, tile, o, p.C, dy);
  };
  if (tiles > 0) {
    load(tiles - 1);
    glr_settle();
  }
  int turn = 0;
  for (int64_t t = tiles - 1; t >= 0; --t, turn ^= 1) {
    const int64_t tile = s.row0 + t * TILE, row = tile + run * ROWS;
    f32x2 state = kept;
    GlrFlags f = {0, 0, 0, ROWS};
    bool slow = false;
    if (FLAT || t == 0 || t == tiles - 1) {
      q.back(p, row);
      slow = __any(glr_flags<ROWS>(p, q, row, s.row1, f));
    }
    // What stays until the gradients: a, the input b = m u, m sigmoid(i), u / m and the
    // gates.  Below the fp32 range m and 1 / m count as 0: u may be of any size there.
    f32x2 a[ROWS], b[ROWS], ms[ROWS], um[ROWS], sr[ROWS], si[ROWS], dv[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const f32x2 rj = to_f2<E>(r[j]), ij = to_f2<E>(i[j]), xj = to_f2<E>(x[j]);
      dv[j] = to_f2<E>(dy[j]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const GlrChannel &k = e ? k1 : k0;
        sr[j][e] = glr_sigmoid(rj[e], k.br);
        si[j][e] = glr_sigmoid(ij[e], k.bi);
        const float l2 = k.k2 * sr[j][e];
        a[j][e] = __builtin_amdgcn_exp2f(l2);
        const float mm = glr_rest(a[j][e], l2), over = mm < 1e-37f ? 0.f : __builtin_amdgcn_rsqf(mm), m = mm * over;
        const float u = si[j][e] * xj[e];
        b[j][e] = m * u;
        ms[j][e] = m * si[j][e];
        um[j][e] = u * over;
      }
    }
    load(t > 0 ? t - 1 : 0);  // behind the last tile that one again
    f32x2 A = {1.f, 1.f}, B = {0.f, 0.f}, Ar = {1.f, 1.f}, G = {0.f, 0.f};
    const auto at = [&](const float *st, int j) {  // row j's sequence of a state
      GlrSeq w = q;
      w.walk(p, row + j);
      return st ? *reinterpret_cast<const f32x2 *>(st + (size_t)w.n * p.C + c) : (f32x2){0.f, 0.f};
    };
    if (slow) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        f32x2 aj = a[j], bj = b[j];
        if (j >= f.live) {
          aj = (f32x2){1.f, 1.f};
          bj = (f32x2){0.f, 0.f};
        } else if (f.dead >> j & 1) {
          aj = (f32x2){GLR_CUT, GLR_CUT};
          bj = (f32x2){0.f, 0.f};
        } else if (f.starts >> j & 1) {
          bj = glr_fma(aj, at(p.h0, j), bj);
          aj = (f32x2){GLR_CUT, GLR_CUT};
        }
        B = glr_map(aj, B, bj);
        A = glr_times(A, aj);
      }
#pragma unroll
      for (int j = ROWS - 1; j >= 0; --j) {
        f32x2 aj = a[j], gj = {a[j][0] * dv[j][0], a[j][1] * dv[j][1]};
        if (j >= f.live) {
          aj = (f32x2){1.f, 1.f};
          gj = (f32x2){0.f, 0.f};
        } else if (f.dead >> j & 1) {
          aj = (f32x2){GLR_CUT, GLR_CUT};
          gj = (f32x2){0.f, 0.f};
        } else if (f.ends >> j & 1) {
          gj = glr_fma(aj, at(p.dhT, j), gj);
          aj = (f32x2){GLR_CUT, GLR_CUT};
        }
        G = glr_map(aj, G, gj);
        Ar = glr_times(Ar, aj);
      }
    } else {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        B = glr_fma(a[j], B, b[j]);
        A = (f32x2){A[0] * a[j][0], A[1] * a[j][1]};
      }
#pragma unroll
      for (int j = ROWS - 1; j >= 0; --j) G = (f32x2){a[j][0] * (dv[j][0] + G[0]), a[j][1] * (dv[j][1] + G[1])};
      Ar = A;
    }
    const f32x2 oA = other_half(A), oB = other_half(B), oAr = other_half(Ar), oG = other_half(G);
    if (!upper) {
      const f32x2 tB = glr_map<FLAT>(oA, B, oB);
      const f32x2 tA = glr_times<FLAT>(A, oA);
      fwd_maps[turn][wave][lane] = (f32x4){tA[0], tA[1], tB[0], tB[1]};
    } else {
      const f32x2 tG = glr_map<FLAT>(oAr, G, oG);
      const f32x2 tA = glr_times<FLAT>(Ar, oAr);
      bwd_maps[turn][wave][lane] = (f32x4){tA[0], tA[1], tG[0], tG[1]};
    }
    __syncthreads();
    f32x4 mf[GLR_WAVES - 1], mb[GLR_WAVES];
#pragma unroll
    for (int k = 0; k < GLR_WAVES - 1; ++k) mf[k] = fwd_maps[turn][k][lane];
#pragma unroll
    for (int k = 0; k < GLR_WAVES; ++k) mb[k] = bwd_maps[turn][k][lane];
#pragma unroll
    for (int k = 0; k < GLR_WAVES - 1; ++k)
      if (k < wave) state = glr_map<FLAT>((f32x2){mf[k][0], mf[k][1]}, state, (f32x2){mf[k][2], mf[k][3]});
    if (upper) state = glr_map<FLAT>(oA, state, oB);
    f32x2 g = {0.f, 0.f};
#pragma unroll
    for (int k = GLR_WAVES - 1; k >= 0; --k) {
      if (k == wave) g = carry;
      carry = glr_map<FLAT>((f32x2){mb[k][0], mb[k][1]}, carry, (f32x2){mb[k][2], mb[k][3]});
    }
    if (!upper) g = glr_map<FLAT>(oAr, g, oG);
    const auto finish = [&](auto slow_c) {
      uint32_t o[ROWS];
      glr_offsets<ROWS>(o, run * ROWS, TILE, pitch, col);
      constexpr bool SLOW = decltype(slow_c)::value;
      f32x2 h[ROWS];  // the state in front of every row
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        if (SLOW && j < f.live && f.starts >> j & 1) state = at(p.h0, j);
        h[j] = state;
        state = glr_fma(a[j], state, b[j]);
      }
#pragma unroll
      for (int j = ROWS - 1; j >= 0; --j) {
        if (SLOW && j >= f.live) continue;
        const bool dead = SLOW && f.dead >> j & 1;
        if (SLOW && f.ends >> j & 1) g = at(p.dhT, j);
        f32x2 dx, dr, di, W;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // W = g log a (a h - u a^2 / m)
          const float ge = dv[j][e] + g[e], la = (e ? k1.k2 : k0.k2) * GLR_LN2 * sr[j][e] * a[j][e], db = ge * b[j][e];
          W[e] = ge * la * __builtin_fmaf(-a[j][e], um[j][e], h[j][e]);
          dr[e] = __builtin_fmaf(-sr[j][e], W[e], W[e]);
          dx[e] = ge * ms[j][e];
          di[e] = __builtin_fmaf(-si[j][e], db, db);
          g[e] = a[j][e] * ge;
        }
        if (SLOW && dead) {
          g = dx = dr = di = (f32x2){0.f, 0.f};
          if (!p.zero_tail) continue;
        } else {
          dlam += W;
          dbr += dr;
          dbi += di;
          if (SLOW && p.dh0 && f.starts >> j & 1) {
            GlrSeq w = q;
            w.walk(p, row + j);
            *reinterpret_cast<f32x2 *>(p.dh0 + (size_t)w.n * p.C + c) = g;
          }
        }
        const auto put = [&](void *out, f32x2 v) { glr_store(glr_base(out, tile * pitch), o[j], to_e2<E>(v)); };
        put(p.dx, dx);
        put(p.dr, dr);
        put(p.di, di);
      }
    };
    if (slow) {
      finish(std::true_type());
      glr_settle();
    } else finish(std::false_type());
  }
  *reinterpret_cast<f32x2 *>(&sums[0][run][2 * lane]) = dlam;
  *reinterpret_cast<f32x2 *>(&sums[1][run][2 * lane]) = dbr;
  *reinterpret_cast<f32x2 *>(&sums[2][run][2 * lane]) = dbi;
  __syncthreads();
  const int which = threadIdx.x / GLR_CH, channel = threadIdx.x % GLR_CH;
  if (which >= 3 || grp * GLR_CH + channel >= p.C) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < GLR_RUNS; ++k) sum += sums[which][k][channel];
  p.part[((size_t)seg * 3 + which) * p.C + grp * GLR_CH + channel] = sum;
}

// The parameters' gradients from the segments' sums.
__global__ __launch_bounds__(ROW_THREADS) void glr_param_kernel(GlrParams p) {
  const int64_t col0 = (int64_t)blockIdx.x * SUM_COLS, n = 3 * (int64_t)p.C, col = col0 + threadIdx.x;
  const float a = column_sum(p.part, p.nseg, n, col0);
  if (threadIdx.x >= SUM_COLS || col >= n) return;
  const int which = (int)(col / p.C), c = (int)(col - (int64_t)which * p.C);
  if (which == 0) {
    // sigmoid(lam) / softplus(lam) is 1 to fp32's last digit where e^lam is below 2^-24
    const float lam = p.lam[c];
    p.dlam[c] = lam < -20.f ? a : a / ((1.f + expf(-lam)) * softplus(lam));
  } else if (which == 1) {
    if (p.dbr) p.dbr[c] = a;
  } else if (p.dbi) {
    p.dbi[c] = a;
  }
}

}  // namespace

hipError_t launch_glr_bwd(const GlrParams &p, int dtype, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.nseg * p.groups)), thr(GLR_THREADS);
  if (dtype == 1) {
    if (p.flat) hipLaunchKernelGGL((glr_bwd_kernel<bf16, BWD_ROWS, true>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((glr_bwd_kernel<bf16, BWD_ROWS, false>), grid, thr, 0, st, p);
  } else {
    if (p.flat) hipLaunchKernelGGL((glr_bwd_kernel<float, BWD_ROWS, true>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((glr_bwd_kernel<float, BWD_ROWS, false>), grid, thr, 0, st, p);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(glr_param_kernel, dim3((unsigned)((3 * (int64_t)p.C + SUM_COLS - 1) / SUM_COLS)), dim3(ROW_THREADS), 0,
                     st, p);
  return hipGetLastError();
}

}  // namespace dn
