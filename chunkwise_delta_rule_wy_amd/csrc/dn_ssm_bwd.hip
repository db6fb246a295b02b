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
// with K and Q are made once for all of them.  dlog's first term is the suffix
// sum of row sums less column sums of E without its diagonal, which belongs to
// no t: where the decay is strong the diagonal outweighs all else, and would
// have to cancel.  The sums are in double, so that what cancels leaves nothing:
// an error there is the same for all earlier tokens and adds up in dA.  Wave (cb, half) = (w % 4, w / 4)
// owns token column block cb of the 64 x 64 matrices, of M and dG only the row
// blocks 2 half, 2 half + 1, and of dv the columns' half; for dq and dk a
// wave owns 16 of the Dk rows.
#include "dn_ssm.h"

namespace dn {
namespace {

constexpr int GRAD_THREADS = 512;

template <int DK>
struct GradLds {
  static constexpr int QS = DK + 8, VS = SSM_TILE + 8, NT = DK / 16;
  alignas(16) bf16 q[CH * QS];
  alignas(16) bf16 k[CH * QS];
  alignas(16) bf16 v[CH * VS];
  alignas(16) bf16 dO[CH * VS];
  alignas(16) bf16 dh[DK * VS];  // dh rounded, for K dh; at the end dG^T
  GateTab tabs[2];               // by the head's parity
  struct Sums {
    double row_x[4][CH], col_x[2][CH], hd[8];
    float col_e[2][CH], diag_e[CH], qd[NT][CH], kd[NT][CH], diag[4];
  } sums[2];
};

template <int DK>
__global__ __launch_bounds__(GRAD_THREADS) void ssm_grad_kernel(SsmParams p) {
  using LD = GradLds<DK>;
  constexpr int KB = DK / 32, QS = LD::QS, VS = LD::VS, NT = LD::NT;
  constexpr int NTT = NT / 2;  // token tiles of a wave's dq and dk
  __shared__ LD s;
  const int w = wave_id(), l = lane_id(), g = l >> 4, m = l & 15;
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
  const int R = p.H / p.G;
  const int h_first = grp * R + set * p.set_heads;
  const int heads = min(p.set_heads, R - set * p.set_heads);
  const int cb = w & 3, half = w >> 2;
  const int n0 = DK == 128 ? 16 * w : 16 * cb, tt0 = DK == 128 ? 0 : 2 * half;
  const bool own_rows = DK == 128 || half == 0;  // one wave per 16 rows of h and dh for their dot product
  const int j = 16 * cb + m;                     // the lane's token column

  {
    Stage<CH, DK, GRAD_THREADS> st;
    const size_t off = (row0 * p.G + grp) * DK, pitch = (size_t)p.G * DK;
    st.load(p.q + off, pitch, L);
    st.template store<QS>(s.q);
    st.load(p.k + off, pitch, L);
    st.template store<QS>(s.k);
  }
  Stage<CH, SSM_TILE, GRAD_THREADS> sv, so;
  f32x4 hr[2][2], dr[2][2];  // the wave's rows of h and dh: [32-column block][half of 8 columns]
  auto fetch = [&](int h, int tile) {
    const size_t off = (row0 * p.H + h) * p.DV + tile * SSM_TILE, pitch = (size_t)p.H * p.DV;
    sv.load(p.v + off, pitch, L);
    so.load(p.dO + off, pitch, L);
    const size_t st = (((size_t)chunk * p.H + h) * DK + n0 + m) * p.DV + tile * SSM_TILE + 8 * g;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        hr[kb][x] = *reinterpret_cast<const f32x4 *>(p.states + st + 32 * kb + 4 * x);
        dr[kb][x] = *reinterpret_cast<const f32x4 *>(p.dstates + st + 32 * kb + 4 * x);
      }
  };
  auto gates = [&](int hh) {  // one wave
    const int h = h_first + hh;
    fill_gates(s.tabs[hh & 1], l < L ? raw_step(p, row0 + l, h) : 0.f, p.A[h], L);
  };
  // the head's sums over the waves and its scalar gradients, by one wave
  auto finish = [&](int hh) {
    const int h = h_first + hh;
    const GateTab &T = s.tabs[hh & 1];
    const typename LD::Sums &x = s.sums[hh & 1];
    float qd = 0.f, kd = 0.f;
    double hd = 0.;
    double db = -(x.col_x[0][l] + x.col_x[1][l]);
    for (int c = 0; c <= (l >> 4); ++c) db += x.row_x[c][l];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      qd += x.qd[t][l];
      kd += x.kd[t][l];
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) hd += x.hd[t];
    const float st = T.s[l], wu = T.w[l] * kd;
    const float ds = ((x.col_e[0][l] + x.col_e[1][l]) + x.diag_e[l]) + wu;
    const double su = (double)st * wu;
    db += (double)(T.gam[l] * qd);
    const double incl = wave_incl_scan_d(db), before = wave_incl_scan_d(su) - su;
    const float dlog = (float)((lane_val_d(incl, 63) - incl + db) + before + (double)T.last * hd);
    const float ddt = (ds + p.A[h] * dlog) * -expm1f(-st);  // sigmoid(x) = 1 - exp(-softplus(x))
    if (l < L) p.ddt[(row0 + l) * p.H + h] = ddt;
    const float dA = wave_sum(st * dlog), db_sum = wave_sum(l < L ? ddt : 0.f);
    if (l == 0) {
      float *out = p.par_part + ((size_t)chunk * p.H + h) * 3;
      out[0] = dA;
      out[1] = db_sum;
      out[2] = (x.diag[0] + x.diag[1]) + (x.diag[2] + x.diag[3]);
    }
  };

  fetch(h_first, 0);
  if (w == 3) gates(0);
  __syncthreads();

  // G: tiles of rows r (four per lane), column j
  f32x4 G[4], dG[2], gm[4];
  bf16x8 kf[KB];  // K row j
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) kf[kb] = frag_row(s.k, QS, j, 32 * kb + 8 * g);
#pragma unroll
  for (int rb = 0; rb < 4; ++rb) {
    G[rb] = zero4();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) G[rb] = mma32(G[rb], frag_row(s.q, QS, 16 * rb + m, 32 * kb + 8 * g), kf[kb]);
  }
  dG[0] = dG[1] = zero4();
  f32x4 dq[NTT], dk[NTT];
#pragma unroll
  for (int t = 0; t < NTT; ++t) dq[t] = dk[t] = zero4();
  const uint32_t aq = lds_addr(s.q), ak = lds_addr(s.k), ao = lds_addr(s.dO), ad = lds_addr(s.dh);

  for (int hh = 0; hh < heads; ++hh) {
    const int h = h_first + hh;
    const GateTab &T = s.tabs[hh & 1];
    typename LD::Sums &sums = s.sums[hh & 1];
    f32x4 M[2];
    M[0] = M[1] = zero4();
    bf16x8 pf[2];
    float sj = 0.f, wsj = 0.f, qd[NTT], kd[NTT];
    double hd = 0.;
#pragma unroll
    for (int t = 0; t < NTT; ++t) qd[t] = kd[t] = 0.f;
    const float skip = p.skip ? p.skip[h] : 0.f;
    for (int tile = 0; tile < p.ntiles; ++tile) {
      __syncthreads();
      sv.template store<VS>(s.v);
      so.template store<VS>(s.dO);
      Split hs[2], ds[2];
      float dot = 0.f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = hr[kb][i >> 2][i & 3];
          y[i] = dr[kb][i >> 2][i & 3];
          dot += x[i] * y[i];
        }
        hs[kb] = split3(x);
        ds[kb] = split3(y);
        if (own_rows) *reinterpret_cast<bf16x8 *>(s.dh + (n0 + m) * VS + 32 * kb + 8 * g) = ds[kb].p[0];
      }
      if (own_rows) hd += (double)dot;
      __syncthreads();
      if (tile + 1 < p.ntiles) fetch(h, tile + 1);
      else if (hh + 1 < heads) fetch(h + 1, 0);
      if (tile == 0) {  // the head's decay ratios and P
        sj = T.s[j];
        wsj = T.ws[j];
        const float bhj = T.bh[j], blj = T.bl[j];
        f32x4 P[4];
#pragma unroll
        for (int rb = 0; rb < 4; ++rb) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 16 * rb + 4 * g + i;
            gm[rb][i] = r >= j ? decay_ratio(T.bh[r], T.bl[r], bhj, blj) : 0.f;
            P[rb][i] = r >= j ? G[rb][i] * gm[rb][i] * sj : 0.f;
          }
        }
        pf[0] = bfrag<bf16>(P[0], P[1]);
        pf[1] = bfrag<bf16>(P[2], P[3]);
      }
      // M, the wave's row blocks
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rb = 2 * half + x;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
          M[x] = mma32(M[x], frag_row(s.dO, VS, 16 * rb + m, 32 * kb + 8 * g), frag_row(s.v, VS, j, 32 * kb + 8 * g));
      }
      // h dO^T and dh V^T, the wave's 16 Dk rows
#pragma unroll
      for (int t = 0; t < NTT; ++t) {
        const int r = 16 * (tt0 + t) + m;
        f32x4 a = zero4(), b = zero4();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const bf16x8 of = frag_row(s.dO, VS, r, 32 * kb + 8 * g), vf = frag_row(s.v, VS, r, 32 * kb + 8 * g);
#pragma unroll
          for (int k = 2; k >= 0; --k) {
            a = mma32(a, hs[kb].p[k], of);
            b = mma32(b, ds[kb].p[k], vf);
          }
        }
        const bf16x4 qv = *reinterpret_cast<const bf16x4 *>(s.q + r * QS + n0 + 4 * g);
        const bf16x4 kv = *reinterpret_cast<const bf16x4 *>(s.k + r * QS + n0 + 4 * g);
        const float gam = T.gam[r], ws = T.ws[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qd[t] += (float)qv[i] * a[i];
          kd[t] += (float)kv[i] * b[i];
          dq[t][i] += gam * a[i];
          dk[t][i] += ws * b[i];
        }
      }
      // dv, token j, the wave's two column tiles
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int pt = 2 * half + x;
        f32x4 a = zero4(), b = zero4();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const int e = (l >> 2) & 3, q4 = l & 3;
          const uint32_t at = ao + (32 * kb + 4 * g + e) * 2 * VS + 2 * (16 * pt + 4 * q4);
          a = mma32(a, wy::cat(wy::ld_tr(at), wy::ld_tr(at + 16 * 2 * VS)), pf[kb]);
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) b = mma32(b, frag_tr(ad, 2 * VS, 32 * kb, 16 * pt), kf[kb]);
        const bf16x4 ov = *reinterpret_cast<const bf16x4 *>(s.dO + j * VS + 16 * pt + 4 * g);
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a[i] + wsj * b[i] + skip * (float)ov[i];
        if (j < L)
          *reinterpret_cast<bf16x4 *>(p.dv + ((row0 + j) * p.H + h) * p.DV + tile * SSM_TILE + 16 * pt + 4 * g) =
              cvt_bf16x4(o);
      }
      if (tile == 0 && w == 3) {  // this wave has no blocks of M below
        if (hh > 0) finish(hh - 1);
        if (hh + 1 < heads) gates(hh + 1);
      }
    }
    // the head's sums over the 64 x 64 matrices
    float col = 0.f, diag = 0.f, diag_e = 0.f;
    double col_x = 0.;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rb = 2 * half + x;
      if (rb < cb) continue;
      const f32x4 gmx = half ? gm[2 + x] : gm[x], Gx = half ? G[2 + x] : G[x];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = 16 * rb + 4 * g + i >= j;
        const float mg = in ? M[x][i] * gmx[i] : 0.f;
        const bool on = rb == cb && 4 * g + i == m;
        float e = in ? mg * Gx[i] : 0.f;
        dG[x][i] += mg * sj;
        if (on) {
          diag = M[x][i];
          diag_e = e;
          e = 0.f;
        }
        col += e;
        const double x64 = (double)(e * sj), row = row_sum16_d(x64);
        col_x += x64;
        if (m == 0) sums.row_x[cb][16 * rb + 4 * g + i] = row;
      }
    }
    col = cross_row_sum(col);
    col_x += __shfl_xor(col_x, 16, 64);
    col_x += __shfl_xor(col_x, 32, 64);
    if (g == 0) {
      sums.col_e[half][j] = col;
      sums.col_x[half][j] = col_x;
    }
    if (half == cb / 2) {
      diag_e = cross_row_sum(diag_e);
      if (g == 0) sums.diag_e[j] = diag_e;
      diag = wave_sum(diag);
      if (l == 0) sums.diag[cb] = diag;
    }
#pragma unroll
    for (int t = 0; t < NTT; ++t) {
      const float a = cross_row_sum(qd[t]), b = cross_row_sum(kd[t]);
      if (g == 0) {
        sums.qd[n0 / 16][16 * (tt0 + t) + m] = a;
        sums.kd[n0 / 16][16 * (tt0 + t) + m] = b;
      }
    }
    hd = row_sum16_d(hd);
    hd += __shfl_xor(hd, 16, 64);
    hd += __shfl_xor(hd, 32, 64);
    if (l == 0) sums.hd[w] = hd;
  }
  __syncthreads();
  if (w == 3) finish(heads - 1);

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
      dq[t] = mma32(dq[t], frag_tr(ak, 2 * QS, 32 * kb, n0), frag_tr(ad, 2 * VS, 32 * kb, 16 * tt));
      dk[t] = mma32(dk[t], frag_tr(aq, 2 * QS, 32 * kb, n0), frag_row(s.dh, VS, r, 32 * kb + 8 * g));
    }
  }
  mfma_settle();
#pragma unroll
  for (int t = 0; t < NTT; ++t) {
    const int r = 16 * (tt0 + t) + m;
    if (r >= L) continue;
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

// Sums over the sets of heads, four elements per thread (blockIdx.y: dq, dk).
constexpr int SUM_THREADS = 256;

__global__ __launch_bounds__(SUM_THREADS) void ssm_set_sum_kernel(SsmParams p, int64_t n4, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * SUM_THREADS + threadIdx.x;
  if (i >= n4) return;
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
    if (p.dq_part) {
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
