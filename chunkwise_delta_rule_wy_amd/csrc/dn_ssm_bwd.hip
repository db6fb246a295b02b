// Selective state space scan, the chunk-parallel part of the backward pass
// (the mathematics of the chunk: dn_ssm.h).  The sweeps have left the state h
// entering every chunk and the gradient dh of the state leaving it, both fp32.
// With M = dO V^T, G = Q K^T, P = G * Gamma * s_j and, per head,
//
//   dq = sum over the group's heads of  dG K + diag(gamma) dO h^T,
//   dk = sum over the group's heads of  dG^T Q + diag(w s) V dh^T,   dG = M * Gamma * s_j
//   dv = P^T dO + diag(w s) K dh + skip dO,
//
// the decays and step sizes, with E = M * G * Gamma,
// u_j = k_j . (dh v_j) and z_r = gamma_r q_r . (h dO_r),
//
//   ds_j   = sum_r E_rj + w_j u_j
//   dlog_t = sum_{j < t <= r} E_rj s_j + sum_{r >= t} z_r + sum_{j < t} s_j w_j u_j + gamma_63 <h, dh>
//   ddt = (ds + A dlog) sigmoid(dt + dt_bias)
//   dA = sum s dlog,   ddt_bias = sum ddt,   dskip = sum_r M_rr.
//
// One workgroup of eight waves owns a chunk of one group and a set of its
// heads: G, dG, dq and dk stay in registers while the heads pass by, so that
// the sum over the heads that share a key costs nothing, and dG's products
// with K and Q are made once for all of them.  dlog's pairs are
// summed as they stand, suffix sums down the columns and then across, never as
// a difference of larger sums: with a strong decay E's diagonal, which belongs
// to no t, outweighs the rest, and an error that all tokens share adds up in
// dA.  Wave (cb, half) owns token column block cb of the 64 x 64 matrices, of M
// and dG only the row blocks 2 half, 2 half + 1, and of dv the columns' half;
// for dq and dk a wave owns 16 of the Dk rows.
//
// 233 registers allow two waves on a SIMD, one workgroup on a CU, so that what
// the next head needs is loaded as soon as its registers are free and without
// a branch.  4 x 4096 tokens, 32 heads of 128 x 64 (256 workgroups): 198 us.
// Neither side bounds it alone: the states, v, dO and dv are 738 MB, 3.7 TB/s
// where a large copy reaches 5.2; without most of the products it takes 188 us,
// without the loads 172 us.  The CU's one workgroup runs loads, LDS and products
// largely one after another, and bank conflicts of the rows, which are padded by
// 16 bytes and not swizzled, take 36 % of its LDS cycles.
#include "dn_ssm.h"

namespace dn {
namespace {

constexpr int GRAD_THREADS = 512;
// Heads between two pauses in which every wave turns one head's sums into its
// scalar gradients and fills one of the next heads' gate tables: both are
// long chains of a few lanes' work, which one wave for each of the two tasks
// beside every head's products would make the kernel's pace (241 against 250
// us, and 183 against 254 us without the loads, before the loads came early).
constexpr int BATCH = GRAD_THREADS / 64;

template <int DK>
struct GradLds {
  static constexpr int QS = DK + 8, VS = SSM_TILE + 8, NT = DK / 16;
  alignas(16) bf16 q[CH * QS];
  alignas(16) bf16 k[CH * QS];
  alignas(16) bf16 v[CH * VS];
  alignas(16) bf16 dO[CH * VS];
  alignas(16) bf16 dh[DK * VS];  // dh rounded, for K dh; at the end dG^T
  alignas(16) bf16 p[CH * VS];   // the head's P^T, zero above the diagonal blocks
  GateTab tabs[BATCH];
  struct Sums {
    double hd[8];
    float pairs[4][CH], col_e[2][CH], diag_e[CH], qd[NT][CH], kd[NT][CH], diag[4];
  } sums[BATCH];
};

template <int DK>
__global__ __launch_bounds__(GRAD_THREADS) void ssm_grad_kernel(SsmParams p) {
  using LD = GradLds<DK>;
  constexpr int KB = DK / 32, QS = LD::QS, VS = LD::VS, NT = LD::NT;
  constexpr int NTT = NT / 2;  // token tiles of a wave's dq and dk
  __shared__ LD s;
  if (p.zero_tail) {
    clear_tail<u32x4>(p, p.dq, (int64_t)p.G * DK / 8);
    clear_tail<u32x4>(p, p.dk, (int64_t)p.G * DK / 8);
    clear_tail<u32x4>(p, p.dv, (int64_t)p.H * p.DV / 8);
    clear_tail<float>(p, p.ddt, p.H);
  }
  const int w = wave_number(), lane = lane_id(), l = lane, g = l >> 4, m = l & 15;
  const int item = xcd_item(blockIdx.x, p.nchunks * p.G * p.sets);
  const int chunk = item / (p.G * p.sets), grp = item % (p.G * p.sets) / p.sets, set = item % p.sets;
  int L;
  size_t row0;
  {
    int n, c, len;
    if (p.cu) {
      n = p.chunk_seq[chunk];
      if (n < 0) return;
      c = chunk - p.chunk_base[n];
      row0 = p.cu[n];
      len = p.cu[n + 1] - p.cu[n];
    } else {
      n = chunk / p.NC;
      c = chunk - n * p.NC;
      row0 = (size_t)n * p.T;
      len = p.T;
    }
    row0 += (size_t)c * CH;
    L = min(CH, len - c * CH);
  }
  // Odd chunks work on -dO and -dh, and their results change sign at the end, so
  // that the one-sided rounding of the matrix products does not add up in dA.
  const uint32_t flip = chunk & 1 ? 0x80008000u : 0u;
  const float sign = chunk & 1 ? -1.f : 1.f;
  const int R = p.H / p.G;
  const int h_first = grp * R + set * p.set_heads;
  const int heads = min(p.set_heads, R - set * p.set_heads);
  const int half = w >> 2, cb = half ? 3 - (w & 3) : w & 3;  // so that the lower blocks are spread over the SIMDs
  const int n0 = DK == 128 ? 16 * w : 16 * cb, tt0 = DK == 128 ? 0 : 2 * half;
  const bool own_rows = DK == 128 || half == 0;  // one wave per 16 rows of h and dh for their dot product
  const int j = 16 * cb + m;                     // the lane's token column

  {
    Stage<CH, DK, GRAD_THREADS> st;
    const size_t off = (row0 * p.G + grp) * DK;
    const uint32_t pitch = 2 * p.G * DK;
    st.load(p.q + off, pitch, L);
    st.template store<QS>(s.q);
    st.load(p.k + off, pitch, L);
    st.template store<QS>(s.k);
  }
  Stage<CH, SSM_TILE, GRAD_THREADS> sv, so;
  f32x4 hr[2][2], dr[2][2], dr_next[2][2];  // the wave's rows of h and dh: [32-column block][half of 8 columns]
  const uint32_t state_off = chunk_state_unit<DK>(n0 / 16, g >> 1, m, 2 * (g & 1));
  auto fetch_rows = [&](int h, int tile) {
    const size_t off = (row0 * p.H + h) * p.DV + tile * SSM_TILE;
    const uint32_t pitch = 2 * p.H * p.DV;
    sv.load_clamped(p.v + off, pitch, L, threadIdx.x);
    so.load_clamped(p.dO + off, pitch, L, threadIdx.x);
  };
  auto fetch_state = [&](const float *states, int h, int tile, f32x4 (&x)[2][2]) {
    const size_t at = ((size_t)chunk * p.H + h) * DK * p.DV + tile * (SSM_TILE * DK);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[kb][i] = ldg<f32x4>(states + at, state_off + chunk_state_unit<DK>(0, 2 * kb, 0, i));
  };
  // the steps and a head's parameters are loaded a batch of heads ahead
  float dt = 0.f, bias = 0.f, A = 0.f, skip_next = 0.f;
  auto load_gates = [&](int hh) {
    const int h = h_first + min(hh, heads - 1);
    dt = load_step(p, row0, L, h);
    A = p.A[h];
    if (p.bias) bias = p.bias[h];
    if (p.skip) skip_next = p.skip[h];
  };
  auto gates = [&](int hh) {
    GateTab &T = s.tabs[hh % BATCH];
    fill_gates(T, dt + bias, A, L);
    if (l == 0) {
      T.A = A;
      T.skip = skip_next;
    }
  };
  // a head's sums over the waves and its scalar gradients
  auto finish = [&](int hh) {
    const int h = h_first + hh;
    const GateTab &T = s.tabs[hh % BATCH];
    const typename LD::Sums &x = s.sums[hh % BATCH];
    float pairs = 0.f, qd = 0.f, kd = 0.f;
    double hd = 0.;
    for (int c = 0; c <= (l >> 4); ++c) pairs += x.pairs[c][l];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      qd += x.qd[t][l];
      kd += x.kd[t][l];
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) hd += x.hd[t];
    const float st = T.s[l], wu = T.w[l] * kd;
    const float ds = ((x.col_e[0][l] + x.col_e[1][l]) + x.diag_e[l]) + wu;
    // sums over the tokens before t, of all and (t < 32) of E's lower rows, and over those from t on
    const double su = (double)st * wu, low = (double)st * x.col_e[1][l], z = (double)(T.gam[l] * qd);
    const double before = wave_incl_scan_d(su) - su, below = wave_incl_scan_d(low) - low;
    const double incl = wave_incl_scan_d(z);
    const double dlog =
        (double)pairs + (l < 32 ? below : 0.) + (lane_val_d(incl, 63) - incl + z) + before + (double)T.last * hd;
    const float ddt = (ds + T.A * (float)dlog) * -expm1f(-st);  // sigmoid(x) = 1 - exp(-softplus(x))
    if (l < L) p.ddt[(row0 + l) * p.H + h] = sign * ddt;
    // the parameters' sums, which all tokens enter, in double from here on
    const double dA_sum = wave_incl_scan_d((double)st * dlog), db_sum = wave_incl_scan_d(l < L ? (double)ddt : 0.);
    if (l == 63) {
      double *out = p.par_part + ((size_t)chunk * p.H + h) * 3;
      out[0] = sign * dA_sum;
      out[1] = sign * db_sum;
      out[2] = sign * (((double)x.diag[0] + x.diag[1]) + ((double)x.diag[2] + x.diag[3]));
    }
  };

  load_gates(w);
  if (w < heads) gates(w);
  fetch_rows(h_first, 0);
  fetch_state(p.states, h_first, 0, hr);
  fetch_state(p.dstates, h_first, 0, dr_next);
  __syncthreads();

  // G: tiles of rows r (four per lane), column j
  f32x4 G[2], dG[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    G[x] = zero4();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
      G[x] = mma32(G[x], frag_row(s.q, QS, 16 * (2 * half + x) + m, 32 * kb + 8 * g), frag_row(s.k, QS, j, 32 * kb + 8 * g));
    *reinterpret_cast<bf16x4 *>(s.p + j * VS + 16 * (2 * half + x) + 4 * g) = cvt_bf16x4(zero4());
  }
  dG[0] = dG[1] = zero4();
  f32x4 dq[NTT], dk[NTT];
#pragma unroll
  for (int t = 0; t < NTT; ++t) dq[t] = dk[t] = zero4();
  const uint32_t aq = lds_addr(s.q), ak = lds_addr(s.k), ao = lds_addr(s.dO), ad = lds_addr(s.dh);

  f32x4 M[2], gm[2];  // M and Gamma of the head, the wave's blocks
  double hd = 0.;
  // A step's rows, dh and, for a head's first tile, P go to LDS (at the end of the
  // step that loads them, which takes 30 registers less than at the start of
  // the next).
  auto stage = [&](int hh, int tile, int l) {
    const int g = l >> 4, m = l & 15, j = 16 * cb + m;
    // dO is zero behind the sequence; v's rows there meet gates of zero
    static_assert(decltype(so)::NU == 1, "one unit a thread");
    so.u[0] = (int)threadIdx.x / decltype(so)::UPR < L ? so.u[0] ^ flip : (u32x4)0u;
#pragma unroll
    for (int x = 0; x < 4; ++x) dr[x >> 1][x & 1] = sign * dr_next[x >> 1][x & 1];
    sv.template store<VS>(s.v);
    so.template store<VS>(s.dO);
    if (own_rows) {
      float dot = 0.f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        *reinterpret_cast<bf16x8 *>(s.dh + (n0 + m) * VS + 32 * kb + 8 * g) = bfrag<bf16>(dr[kb][0], dr[kb][1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot += hr[kb][i >> 2][i & 3] * dr[kb][i >> 2][i & 3];
      }
      hd = tile == 0 ? (double)dot : hd + (double)dot;
    }
    if (tile == 0) {
      const GateTab &T = s.tabs[hh % BATCH];
      const float bhj = T.bh[j], blj = T.bl[j], sj = T.s[j];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rb = 2 * half + x, r0 = 16 * rb + 4 * g;
        if (rb < cb) continue;
        gm[x] = decay_ratios(T, r0, bhj, blj, 1.f);
        f32x4 P;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = computed(G[x][i] * (gm[x][i] * sj));
          P[i] = r0 + i >= j ? v : 0.f;
        }
        *reinterpret_cast<bf16x4 *>(s.p + j * VS + r0) = cvt_bf16x4(P);
      }
    }
    __syncthreads();
  };
  gm[0] = gm[1] = zero4();
  stage(0, 0, l);
  // over the heads and their tiles, in one loop: with one in the other, what a
  // step loads for the next would be copied, and waited for, in between
  for (int hh = 0, tile = 0;;) {
    const int h = h_first + hh, place = hh % BATCH;
    const GateTab &T = s.tabs[place];
    typename LD::Sums &sums = s.sums[place];
    // what the next step needs (the last step loads its own again: a load that
    // may not take place would hold two sets of registers)
    const bool next_tile = tile + 1 < p.ntiles, more = next_tile || hh + 1 < heads;
    const int nh = next_tile || !more ? h : h + 1, nt = next_tile ? tile + 1 : more ? 0 : tile;
    if (tile == 0) M[0] = M[1] = zero4();
    const int l = fresh(lane), g = l >> 4, m = l & 15, j = 16 * cb + m;
    if (tile == 0 && place == 0) load_gates(hh + BATCH + w);
    fetch_rows(nh, nt);
    fetch_state(p.dstates, nh, nt, dr_next);
    // h dO^T, then dh V^T: the wave's 16 Dk rows.  h's registers are free after
    // that for the next one, which arrives during the rest.
    auto rows = [&](const f32x4 (&st)[2][2], const bf16 *ly, const bf16 *lx, const float *coef, f32x4 (&acc)[NTT],
                    float *dots) {
      f32x4 a[NTT];
#pragma unroll
      for (int t = 0; t < NTT; ++t) a[t] = zero4();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        bf16x8 y[NTT];
#pragma unroll
        for (int t = 0; t < NTT; ++t) y[t] = frag_row(ly, VS, 16 * (tt0 + t) + m, 32 * kb + 8 * g);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = st[kb][i >> 2][i & 3];
        const Split sp = split3(x);
#pragma unroll
        for (int k = 2; k >= 0; --k)
#pragma unroll
          for (int t = 0; t < NTT; ++t) a[t] = mma32(a[t], sp.p[k], y[t]);
      }
      float dot[NTT];
#pragma unroll
      for (int t = 0; t < NTT; ++t) {
        const int r = 16 * (tt0 + t) + m;
        const bf16x4 xv = *reinterpret_cast<const bf16x4 *>(lx + r * QS + n0 + 4 * g);
        const float c = coef[r];
        dot[t] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot[t] += (float)xv[i] * a[t][i];
          acc[t][i] += c * a[t][i];
        }
      }
      const float sum = rows_sums(dot);
      if (g < NTT) {
        float *d = dots + 16 * (tt0 + g) + m;
        *d = tile == 0 ? sum : *d + sum;
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    rows(hr, s.dO, s.q, T.gam, dq, sums.qd[n0 / 16]);
    fetch_state(p.states, nh, nt, hr);
    rows(dr, s.v, s.k, T.ws, dk, sums.kd[n0 / 16]);
    // M, the wave's row blocks
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const bf16x8 vf = frag_row(s.v, VS, j, 32 * kb + 8 * g);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        M[x] = mma32(M[x], frag_row(s.dO, VS, 16 * (2 * half + x) + m, 32 * kb + 8 * g), vf);
    }
    __builtin_amdgcn_sched_barrier(0);
    // dv, token j, the wave's two column tiles
    {
      f32x4 a[2], b[2];
      a[0] = a[1] = b[0] = b[1] = zero4();
      const float wsj = T.ws[j], skip = T.skip;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (2 * kb + 1 < cb) continue;  // zeros
        const bf16x8 pf = frag_row(s.p, VS, j, 32 * kb + 8 * g);
#pragma unroll
        for (int x = 0; x < 2; ++x) a[x] = mma32(a[x], frag_tr(ao, 2 * VS, 32 * kb, 16 * (2 * half + x), l), pf);
      }
      mfma_settle();
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const bf16x8 kf = frag_row(s.k, QS, j, 32 * kb + 8 * g);
#pragma unroll
        for (int x = 0; x < 2; ++x) b[x] = mma32(b[x], frag_tr(ad, 2 * VS, 32 * kb, 16 * (2 * half + x), l), kf);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = 16 * (2 * half + x) + 4 * g;
        const bf16x4 ov = *reinterpret_cast<const bf16x4 *>(s.dO + j * VS + c);
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = sign * (a[x][i] + wsj * b[x][i] + skip * (float)ov[i]);
        if (j < L)
          stg<bf16x4>(p.dv + (row0 * p.H + h) * p.DV + tile * SSM_TILE, 2 * (j * (p.H * p.DV) + c), cvt_bf16x4(o));
      }
    }
    if (!next_tile) {
      // the head's sums over the 64 x 64 matrices; `below` sums a column's rows
      // after the tile
      const float sj = T.s[j];
      float below = 0.f, diag = 0.f, diag_e = 0.f;
#pragma unroll
      for (int x = 1; x >= 0; --x) {
        const int rb = 2 * half + x, r0 = 16 * rb + 4 * g;
        if (rb < cb) continue;
        f32x4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = computed(M[x][i] * gm[x][i]);
          dG[x][i] += (r0 + i >= j ? v : 0.f) * sj;
          const float u = computed(v * G[x][i]);
          e[i] = r0 + i > j ? u : 0.f;
          diag = r0 + i == j ? M[x][i] : diag;
          diag_e = r0 + i == j ? u : diag_e;
        }
        // over the rows from this one on
        e[2] += e[3];
        e[1] += e[2];
        e[0] += e[1];
        float after;
        const float sum = row_suffix(e[0], g, after);
        after += below;
        below += sum;
        f32x4 d;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = r0 + i > j ? (e[i] + after) * sj : 0.f;
        const float sums_m = row_sums16(d, m);
        if (m < 4) sums.pairs[cb][r0 + m] = sums_m;
        __builtin_amdgcn_sched_barrier(0);
      }
      if (g == 0) sums.col_e[half][j] = below;
      if (half == cb / 2) {
        diag_e = cross_row_sum(diag_e);
        if (g == 0) sums.diag_e[j] = diag_e;
        diag = wave_sum(diag);
        if (l == 0) sums.diag[cb] = diag;
      }
      hd = row_sum16_d(hd);
      hd += __shfl_xor(hd, 16, 64);
      hd += __shfl_xor(hd, 32, 64);
      if (l == 0) sums.hd[w] = hd;
      if (place == BATCH - 1 || hh + 1 == heads) {
        __syncthreads();
        if (w <= place) finish(hh - place + w);
        if (hh + 1 + w < heads) gates(hh + 1 + w);
      }
    }
    if (!more) break;
    hh += next_tile ? 0 : 1;
    tile = nt;
    __syncthreads();
    stage(hh, tile, fresh(lane));
  }

  // dG^T into LDS (rows j, row blocks above the diagonal zero), then its
  // products with K and Q
#pragma unroll
  for (int x = 0; x < 2; ++x)
    *reinterpret_cast<bf16x4 *>(s.dh + j * VS + 16 * (2 * half + x) + 4 * g) = cvt_bf16x4(dG[x]);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NTT; ++t) {
    const int tt = tt0 + t, r = 16 * tt + m;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      dq[t] = mma32(dq[t], frag_tr(ak, 2 * QS, 32 * kb, n0, l), frag_tr(ad, 2 * VS, 32 * kb, 16 * tt, l));
      dk[t] = mma32(dk[t], frag_tr(aq, 2 * QS, 32 * kb, n0, l), frag_row(s.dh, VS, r, 32 * kb + 8 * g));
    }
  }
  mfma_settle();
#pragma unroll
  for (int t = 0; t < NTT; ++t) {
    const int r = 16 * (tt0 + t) + m;
    if (r >= L) continue;
    dq[t] *= sign;
    dk[t] *= sign;
    const size_t at = ((row0 + r) * p.G + grp) * DK + n0 + 4 * g;
    if (p.dq_part) {
      const size_t part = (size_t)set * p.rows * p.G * DK + at;
      *reinterpret_cast<f32x4 *>(p.dq_part + part) = dq[t];
      *reinterpret_cast<f32x4 *>(p.dk_part + part) = dk[t];
    } else {
      *reinterpret_cast<bf16x4 *>(p.dq + at) = cvt_bf16x4(dq[t]);
      *reinterpret_cast<bf16x4 *>(p.dk + at) = cvt_bf16x4(dk[t]);
    }
  }
}

// Sums over the sets of heads, four elements per thread (blockIdx.y: dq, dk);
// rows behind the last packed sequence have none and stay as they are.
constexpr int SUM_THREADS = 256;

__global__ __launch_bounds__(SUM_THREADS) void ssm_set_sum_kernel(SsmParams p, int64_t n4, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * SUM_THREADS + threadIdx.x;
  if (i >= (p.cu ? n4 / p.rows * p.cu[p.N] : n4)) return;
  const float *src = (blockIdx.y ? p.dk_part : p.dq_part) + 4 * i;
  f32x4 a = *reinterpret_cast<const f32x4 *>(src);
  for (int k = 1; k < p.sets; ++k) a += *reinterpret_cast<const f32x4 *>(src + k * n);
  *reinterpret_cast<bf16x4 *>((blockIdx.y ? p.dk : p.dq) + 4 * i) = cvt_bf16x4(a);
}

// Sums of the per-chunk parameter gradients, one workgroup per head, in double
// and in a fixed order.
__global__ __launch_bounds__(SUM_THREADS) void ssm_param_sum_kernel(SsmParams p) {
  __shared__ double part[SUM_THREADS][3];
  const int h = blockIdx.x, t = threadIdx.x;
  const int n = p.cu ? p.chunk_base[p.N] : p.nchunks;
  double a[3] = {0., 0., 0.};
  for (int c = t; c < n; c += SUM_THREADS)
#pragma unroll
    for (int i = 0; i < 3; ++i) a[i] += p.par_part[((size_t)c * p.H + h) * 3 + i];
#pragma unroll
  for (int i = 0; i < 3; ++i) part[t][i] = a[i];
  for (int d = SUM_THREADS / 2; d > 0; d >>= 1) {
    __syncthreads();
    if (t < d)
#pragma unroll
      for (int i = 0; i < 3; ++i) part[t][i] += part[t + d][i];
  }
  if (t == 0) {
    p.dA[h] = (float)part[0][0];
    if (p.ddt_bias) p.ddt_bias[h] = (float)part[0][1];
    if (p.dskip) p.dskip[h] = (float)part[0][2];
  }
}

}  // namespace

hipError_t launch_ssm_grad(const SsmParams &p, int DK, hipStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)p.nchunks * p.G * p.sets);
  if (grid > 0) {
    if (DK == 64) hipLaunchKernelGGL((ssm_grad_kernel<64>), dim3(grid), dim3(GRAD_THREADS), 0, stream, p);
    else hipLaunchKernelGGL((ssm_grad_kernel<128>), dim3(grid), dim3(GRAD_THREADS), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.dq_part && p.rows > 0) {
      const int64_t n = p.rows * p.G * DK, n4 = n / 4;
      hipLaunchKernelGGL(ssm_set_sum_kernel, dim3((unsigned)((n4 + SUM_THREADS - 1) / SUM_THREADS), 2),
                         dim3(SUM_THREADS), 0, stream, p, n4, n);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  hipLaunchKernelGGL(ssm_param_sum_kernel, dim3(p.H), dim3(SUM_THREADS), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dn
