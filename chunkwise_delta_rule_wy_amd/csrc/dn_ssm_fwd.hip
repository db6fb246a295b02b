// Selective state space scan, forward pass, and the sweeps that the forward
// and the backward pass share (the mathematics: dn_ssm.h).
//
// One workgroup of four waves owns one (segment, head, 64 Dv columns); wave w
// keeps its Dk x 16 slice of the state in registers and the segment's chunks
// pass through LDS, the next chunk's rows already on their way into registers.
#include "dn_ssm.h"

namespace dn {
namespace {

// ------------------------------------------------------------------ sweep
//
// S <- gamma_63 S + X^T diag(c) Y over a segment's chunks, c scaling Y.  The
// accumulators hold S^T tiles (rows: the wave's 16 Dv columns, columns: Dk),
// so that a lane's four rows are 16 consecutive bytes of the stored state.
// Without STORE the sweep starts from zero and leaves the segment's own end
// state (`seg_state`) and log decay; with it, it starts from the joined state
// and stores the state of every chunk before the chunk's update.  REV runs
// the chunks backwards over (q, dO, gamma).  The accumulators change sign from
// chunk to chunk: the matrix instructions' sums come out below the exact ones
// on average (by some 2^-25 of their size), and an error of one sign in the
// states would add up in dA, where it reached 2e-6 of the result.
template <int DK>
struct SweepLds {
  static constexpr int XS = DK + 16, YS = SSM_TILE + 16;  // row strides: 4 rows of a transposed read in separate banks
  alignas(16) bf16 x[CH * XS];
  alignas(16) bf16 y[CH * YS];
  GateTab tabs[2];
};

template <int DK, bool REV, bool STORE>
__device__ __forceinline__ void sweep(const SsmParams &p, SweepLds<DK> &lds, int item) {
  constexpr int XS = SweepLds<DK>::XS, YS = SweepLds<DK>::YS;
  constexpr int NT = DK / 16;
  const int per = p.H * p.ntiles;
  const int seg = item / per, h = item % per / p.ntiles, tile = item % p.ntiles;
  Segment sg;
  if (!segment(p, seg, sg)) return;
  if (!STORE && (REV ? sg.first : sg.last)) return;  // nothing follows it
  const int w = wave_number(), l = lane_id(), g = l >> 4, m = l & 15;
  const int grp = h / (p.H / p.G);
  const bf16 *X = (REV ? p.q : p.k) + (sg.row * p.G + grp) * DK;
  const bf16 *Y = (REV ? p.dO : p.v) + (sg.row * p.H + h) * p.DV + tile * SSM_TILE;
  const size_t xp = (size_t)p.G * DK, yp = (size_t)p.H * p.DV;  // elements of a token
  const int nch = (sg.len + CH - 1) / CH;
  const size_t per_state = (size_t)DK * p.DV;
  // byte offsets of the lane's four columns in the state's row m, and of 16 rows
  const uint32_t lane_off = 4 * (m * p.DV + tile * SSM_TILE + 16 * w + 4 * g), rows16 = 64 * p.DV;
  const float A = p.A[h];

  f32x4 S[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) S[t] = zero4();
  if (STORE) {
    const float *src = p.split ? p.seg_state[REV] + ((size_t)seg * p.H + h) * per_state
                               : (REV ? p.dhT : p.h0);
    if (src) {
      if (!p.split) src += ((size_t)sg.n * p.H + h) * per_state;
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t] = ldg<f32x4>(src, lane_off + t * rows16);
    }
  }

  Stage<CH, DK, NTHR> sx;
  Stage<CH, SSM_TILE, NTHR> sy;
  auto at = [&](int i) { return REV ? nch - 1 - i : i; };
  auto fetch = [&](int c) {
    const int L = min(CH, sg.len - c * CH);
    sx.load(X + c * (CH * xp), 2 * (uint32_t)xp, L);
    sy.load(Y + c * (CH * yp), 2 * (uint32_t)yp, L);
  };
  double logd = 0.;
  float sign = 1.f;  // of the accumulators
  auto gates = [&](int i) {  // one wave
    const int c = at(i), L = min(CH, sg.len - c * CH);
    const float raw = l < L ? raw_step(p, sg.row + (size_t)c * CH + l, h) : 0.f;
    logd += fill_gates(lds.tabs[i & 1], raw, A, L);
  };
  fetch(at(0));
  if (w == 0) gates(0);
  const uint32_t ax = lds_addr(lds.x), ay = lds_addr(lds.y);
  for (int i = 0; i < nch; ++i) {
    const int c = at(i);
    __syncthreads();
    sx.template store<SweepLds<DK>::XS>(lds.x);
    sy.template store<SweepLds<DK>::YS>(lds.y);
    __syncthreads();
    if (i + 1 < nch) fetch(at(i + 1));
    const GateTab &T = lds.tabs[i & 1];
    if (STORE) {
      float *dst = (REV ? p.dstates : p.states) + ((size_t)chunk_id(p, sg, c) * p.H + h) * per_state;
#pragma unroll
      for (int t = 0; t < NT; ++t) stg<f32x4>(dst, lane_off + t * rows16, sign * S[t]);
    }
    sign = -sign;
    Split ysp[2];
    const float *coef = REV ? T.gam : T.ws;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float y[8];
      unpack8(frag_tr(ay, 2 * YS, 32 * kb, 16 * w, l), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= sign * coef[32 * kb + 8 * g + e];
      ysp[kb] = split3(y);
    }
    const float last = T.last;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 acc = S[t] * -last;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 x = frag_tr(ax, 2 * XS, 32 * kb, 16 * t, l);
#pragma unroll
        for (int k = 2; k >= 0; --k) acc = mma32(acc, ysp[kb].p[k], x);
      }
      S[t] = acc;
    }
    if (w == 0 && i + 1 < nch) gates(i + 1);
  }
  float *dst = nullptr;
  if (!STORE) {
    dst = p.seg_state[REV] + ((size_t)seg * p.H + h) * per_state;
    if (tile == 0 && threadIdx.x == 0) p.seg_decay[(size_t)seg * p.H + h] = logd;
  } else if (REV && sg.first && p.dh0) {
    dst = p.dh0 + ((size_t)sg.n * p.H + h) * per_state;
  }
  if (dst) {
    mfma_settle();
#pragma unroll
    for (int t = 0; t < NT; ++t) stg<f32x4>(dst, lane_off + t * rows16, sign * S[t]);
  }
}

// items of both directions: the forward sweep's first, then the reverse one's
template <int DK, bool STORE>
__global__ __launch_bounds__(NTHR) void ssm_sweep_kernel(SsmParams p) {
  const int total = p.nseg * p.H * p.ntiles;
  const int item = xcd_item(blockIdx.x, total);
  __shared__ SweepLds<DK> lds;
  if (blockIdx.y == 0)
    sweep<DK, false, STORE>(p, lds, item);
  else
    sweep<DK, true, STORE>(p, lds, item);
}

// ------------------------------------------------------------------- join
//
// Start states of a sequence's segments from their own end states and decays,
// in place, four state elements per thread; a sequence without tokens hands
// its initial state on.  Bound by the segment states' traffic.
constexpr int JOIN_THREADS = 256;

__global__ __launch_bounds__(JOIN_THREADS) void ssm_join_kernel(SsmParams p, int dk) {
  const bool rev = blockIdx.y == 1;
  const size_t per = (size_t)dk * p.DV;
  const int blocks = (int)(per / (4 * JOIN_THREADS));
  const int nh = blockIdx.x / blocks;
  const int n = nh / p.H, h = nh % p.H;
  const size_t e = (size_t)(blockIdx.x % blocks) * 4 * JOIN_THREADS + 4 * threadIdx.x;
  int s0, cnt;
  if (p.cu) {
    s0 = p.seg_base[n];
    cnt = p.seg_base[n + 1] - s0;
  } else {
    s0 = n * p.NS;
    cnt = p.NS;
  }
  const float *init = rev ? p.dhT : p.h0;
  f32x4 cur = init ? *reinterpret_cast<const f32x4 *>(init + (size_t)nh * per + e) : zero4();
  float *st = p.seg_state[rev];
  for (int i = 0; i < cnt; ++i) {
    const size_t at = (size_t)(rev ? s0 + cnt - 1 - i : s0 + i) * p.H + h;
    f32x4 *x = reinterpret_cast<f32x4 *>(st + at * per + e);
    if (i + 1 == cnt) {  // no sweep has filled this one
      *x = cur;
      break;
    }
    const f32x4 own = *x;
    *x = cur;
    const float d = (float)exp2(p.seg_decay[at]);
    cur = cur * d + own;
  }
  float *out = rev ? p.dh0 : p.hT;
  if (cnt == 0 && out) *reinterpret_cast<f32x4 *>(out + (size_t)nh * per + e) = cur;
}

// ---------------------------------------------------------------- forward
//
// Per chunk: the lower 16 x 16 blocks of P = ((Q K^T) * Gamma) diag(s) (wave w
// computes row block w, rounded to bf16 into LDS), then every wave's 16
// columns of O^T = V^T P^T + diag(gamma) h^T Q^T and of the state update.  The
// state tiles hold Dk rows in the order prow, so that two stacked tiles are
// the operand of h^T Q^T.  While the other waves compute P, wave 0, whose row
// block is the shortest, fills the next chunk's gate table.
template <int DK>
struct FwdLds {
  static constexpr int QS = DK + 8, KS = DK + 8, VS = SSM_TILE + 16, PS = CH + 8;
};

template <int DK>
__global__ __launch_bounds__(NTHR, 2) void ssm_fwd_kernel(SsmParams p) {
  using LD = FwdLds<DK>;
  constexpr int MT = DK / 16, KB = DK / 32;
  __shared__ __align__(16) bf16 lq[CH * LD::QS];
  __shared__ __align__(16) bf16 lk[CH * LD::KS];
  __shared__ __align__(16) bf16 lv[CH * LD::VS];
  __shared__ __align__(16) bf16 lp[CH * LD::PS];
  __shared__ GateTab tabs[2];
  const int per = p.H * p.ntiles;
  const int item = xcd_item(blockIdx.x, p.nseg * per);
  const int seg = item / per, h = item % per / p.ntiles, tile = item % p.ntiles;
  Segment sg;
  if (!segment(p, seg, sg)) return;
  const int w = wave_number(), l = lane_id(), g = l >> 4, m = l & 15;
  const int grp = h / (p.H / p.G);
  const bf16 *Q = p.q + (sg.row * p.G + grp) * DK, *K = p.k + (sg.row * p.G + grp) * DK;
  const size_t vo = (sg.row * p.H + h) * p.DV + tile * SSM_TILE;
  const bf16 *V = p.v + vo;
  bf16 *O = p.o + vo;
  const size_t kp = (size_t)p.G * DK, vp = (size_t)p.H * p.DV;
  const int nch = (sg.len + CH - 1) / CH;
  const size_t per_state = (size_t)DK * p.DV;
  const int col = tile * SSM_TILE + 16 * w + m;
  const float A = p.A[h], skip = p.skip ? p.skip[h] : 0.f;

  f32x4 S[MT];  // rows prow(mt, 4 g + i), column m of the wave's 16
  const float *src = p.split ? p.seg_state[0] + ((size_t)seg * p.H + h) * per_state
                             : (p.h0 ? p.h0 + ((size_t)sg.n * p.H + h) * per_state : nullptr);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) S[t][i] = src ? ldg<float>(src, 4 * (prow(t, 4 * g + i) * p.DV + col)) : 0.f;

  Stage<CH, DK, NTHR> sq, sk;
  Stage<CH, SSM_TILE, NTHR> sv;
  auto fetch = [&](int c) {
    const int L = min(CH, sg.len - c * CH);
    sq.load(Q + c * (CH * kp), 2 * (uint32_t)kp, L);
    sk.load(K + c * (CH * kp), 2 * (uint32_t)kp, L);
    sv.load(V + c * (CH * vp), 2 * (uint32_t)vp, L);
  };
  auto gates = [&](int c) {  // one wave
    const int L = min(CH, sg.len - c * CH);
    const float raw = l < L ? raw_step(p, sg.row + (size_t)c * CH + l, h) : 0.f;
    fill_gates(tabs[c & 1], raw, A, L);
  };
  if (nch > 0) fetch(0);
  if (w == 0 && nch > 0) gates(0);
  const uint32_t ak = lds_addr(lk), av = lds_addr(lv);
  for (int c = 0; c < nch; ++c) {
    const int L = min(CH, sg.len - c * CH);
    __syncthreads();
    sq.template store<LD::QS>(lq);
    sk.template store<LD::KS>(lk);
    sv.template store<LD::VS>(lv);
    __syncthreads();
    if (c + 1 < nch) fetch(c + 1);
    const GateTab &T = tabs[c & 1];

    // P, row block w: tiles hold rows j (four per lane), column r
    {
      const int r = 16 * w + m;
      bf16x8 qf[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) qf[kb] = frag_row(lq, LD::QS, r, 32 * kb + 8 * g);
      const float bhr = T.bh[r], blr = T.bl[r];
      const int nb = (w | 1) + 1;  // whole 32-token blocks
      for (int jb = 0; jb < nb; ++jb) {
        f32x4 acc = zero4();
        if (jb <= w) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) acc = mma32(acc, frag_row(lk, LD::KS, 16 * jb + m, 32 * kb + 8 * g), qf[kb]);
        }
        mfma_settle();
        const int j0 = 16 * jb + 4 * g;
        const f32x4 gm = decay_ratios(T, j0, bhr, blr, -1.f), sj = lds4(T.s + j0);
        f32x4 pr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = computed(acc[i] * (gm[i] * sj[i]));
          pr[i] = j0 + i <= r ? x : 0.f;
        }
        *reinterpret_cast<bf16x4 *>(lp + r * LD::PS + 16 * jb + 4 * g) = cvt_bf16x4(pr);
      }
    }
    if (w == 0 && c + 1 < nch) gates(c + 1);
    __syncthreads();

    // O^T tiles: rows the wave's 16 columns, column r
    bf16x8 vf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) vf[kb] = frag_tr(av, 2 * LD::VS, 32 * kb, 16 * w, l);
    bf16x8 sf[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) sf[kb] = bfrag<bf16>(S[2 * kb], S[2 * kb + 1]);
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      const int r = 16 * rb + m;
      f32x4 a = zero4(), b = zero4();
#pragma unroll
      for (int kb = 0; kb <= rb / 2; ++kb) a = mma32(a, vf[kb], frag_row(lp, LD::PS, r, 32 * kb + 8 * g));
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) b = mma32(b, sf[kb], frag_row(lq, LD::QS, r, 32 * kb + 8 * g));
      const bf16x4 vr = *reinterpret_cast<const bf16x4 *>(lv + r * LD::VS + 16 * w + 4 * g);
      const float gam = T.gam[r];
      f32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = a[i] + gam * b[i] + skip * (float)vr[i];
      if (r < L) stg<bf16x4>(O + c * (CH * vp), 2 * (r * (uint32_t)vp + 16 * w + 4 * g), cvt_bf16x4(o));
    }

    // state update
    Split vsp[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float x[8];
      unpack8(vf[kb], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= T.ws[32 * kb + 8 * g + e];
      vsp[kb] = split3(x);
    }
    const float last = T.last;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      f32x4 acc = S[t] * last;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        // K^T rows in the order prow
        const int e = (l >> 2) & 3, q4 = l & 3;
        const uint32_t a = ak + (32 * kb + 8 * g + e) * 2 * LD::KS + 2 * prow(t, 4 * q4);
        const bf16x8 kf = wy::cat(wy::ld_tr(a), wy::ld_tr(a + 8 * LD::KS));
#pragma unroll
        for (int k = 2; k >= 0; --k) acc = mma32(acc, kf, vsp[kb].p[k]);
      }
      S[t] = acc;
    }
  }
  if (p.hT && sg.last) {
    mfma_settle();
    float *dst = p.hT + ((size_t)sg.n * p.H + h) * per_state;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) stg<float>(dst, 4 * (prow(t, 4 * g + i) * p.DV + col), S[t][i]);
  }
}

}  // namespace

hipError_t launch_ssm_sweep(const SsmParams &p, int DK, bool store, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.nseg * p.H * p.ntiles), backward ? 2 : 1);
  if (grid.x == 0) return hipSuccess;
  if (DK == 64) {
    if (store) hipLaunchKernelGGL((ssm_sweep_kernel<64, true>), grid, dim3(NTHR), 0, stream, p);
    else hipLaunchKernelGGL((ssm_sweep_kernel<64, false>), grid, dim3(NTHR), 0, stream, p);
  } else {
    if (store) hipLaunchKernelGGL((ssm_sweep_kernel<128, true>), grid, dim3(NTHR), 0, stream, p);
    else hipLaunchKernelGGL((ssm_sweep_kernel<128, false>), grid, dim3(NTHR), 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_ssm_join(const SsmParams &p, int DK, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.N * p.H * DK * p.DV / (4 * JOIN_THREADS)), backward ? 2 : 1);
  hipLaunchKernelGGL(ssm_join_kernel, grid, dim3(JOIN_THREADS), 0, stream, p, DK);
  return hipGetLastError();
}

hipError_t launch_ssm_fwd(const SsmParams &p, int DK, hipStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)p.nseg * p.H * p.ntiles);
  if (grid == 0) return hipSuccess;
  if (DK == 64) hipLaunchKernelGGL((ssm_fwd_kernel<64>), dim3(grid), dim3(NTHR), 0, stream, p);
  else hipLaunchKernelGGL((ssm_fwd_kernel<128>), dim3(grid), dim3(NTHR), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dn
