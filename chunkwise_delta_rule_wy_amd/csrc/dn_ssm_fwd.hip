// Selective state space scan, forward pass, and the sweeps that the forward
// and the backward pass share (the mathematics: dn_ssm.h).
//
// One workgroup owns one segment and 64 columns of one head (four waves), or
// twice 64 (SsmPair, eight waves); a wave keeps a Dk x 16 slice of the state in
// registers, and the segment's chunks pass through LDS, the next chunk's rows
// already on their way into registers.
#include "dn_ssm.h"

namespace dn {
namespace {

// What a workgroup works on: `head` and `tile` of each of its SUBS halves.
template <int PAIR>
struct Work {
  static constexpr int SUBS = PAIR == SSM_SINGLE ? 1 : 2, TABS = PAIR == SSM_HEADS ? 2 : 1;
  static constexpr int THREADS = 256 * SUBS;
  int seg, head[SUBS], col[SUBS];  // col: the half's first column
  __device__ __forceinline__ Work(const SsmParams &p, int item) {
    const int per_head = PAIR == SSM_TILES ? p.ntiles / 2 : p.ntiles;  // items
    const int heads = PAIR == SSM_HEADS ? p.H / 2 : p.H;
    const int per = heads * per_head;
    seg = item / per;
    const int x = item - seg * per, h = x / per_head, t = x - h * per_head;
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      head[i] = PAIR == SSM_HEADS ? 2 * h + i : h;
      col[i] = SSM_TILE * (PAIR == SSM_TILES ? 2 * t + i : t);
    }
  }
};
int work_items(const SsmParams &p) {
  const int64_t n = (int64_t)p.nseg * p.H * p.ntiles;
  return (int)(p.pair == SSM_SINGLE ? n : n / 2);
}

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
//
// Measured at 4 x 4096 tokens, 32 heads of 128 x 64: without STORE 37 us
// forwards (8 segments a sequence) and 62 us both ways (4 segments), bound by
// issue (a SIMD issues matrix and vector instructions by turns: 260 vector
// ones a chunk, half of them split3, beside 48 products); with STORE both ways 136 us, 537 MB of
// states and 150 MB of inputs at 5.1 TB/s.
template <int DK, int PAIR>
struct SweepLds {
  static constexpr int YC = SSM_TILE * Work<PAIR>::SUBS;
  alignas(256) bf16 x[CH * DK];
  alignas(256) bf16 y[CH * YC];
  GateTab tabs[2][Work<PAIR>::TABS];
};

template <int DK, int PAIR, bool REV, bool STORE>
__device__ __forceinline__ void sweep(const SsmParams &p, SweepLds<DK, PAIR> &lds, int item) {
  using WK = Work<PAIR>;
  using XT = Swz<DK>;
  using YT = Swz<SweepLds<DK, PAIR>::YC>;
  constexpr int NT = DK / 16, SUBS = WK::SUBS, TABS = WK::TABS, YC = SweepLds<DK, PAIR>::YC;
  const WK wk(p, item);
  Segment sg;
  if (!segment(p, wk.seg, sg)) return;
  if (!STORE && (REV ? sg.first : sg.last)) return;  // nothing follows it
  const int w = wave_number(), l = lane_id(), g = l >> 4, m = l & 15;
  const int sub = SUBS == 2 ? w >> 2 : 0, head = sub ? wk.head[SUBS - 1] : wk.head[0];
  const int col = (sub ? wk.col[SUBS - 1] : wk.col[0]) + 16 * (w & 3);  // the wave's first column
  const int grp = wk.head[0] / (p.H / p.G);
  const size_t xp = (size_t)p.G * DK, yp = (size_t)p.H * p.DV;  // elements of a token
  const bf16 *X = (REV ? p.q : p.k) + sg.row * xp + (size_t)grp * DK;
  const bf16 *Y = (REV ? p.dO : p.v) + sg.row * yp;
  const int nch = (sg.len + CH - 1) / CH;
  const size_t per_state = (size_t)DK * p.DV;
  // byte offsets of the lane's four columns in the state's row m, and of 16 rows
  const uint32_t lane_off = 4 * (m * p.DV + 4 * g), rows16 = 64 * p.DV;

  f32x4 S[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) S[t] = zero4();
  if (STORE) {
    const float *src = p.split ? p.seg_state[REV] : (REV ? p.dhT : p.h0);
    if (src) {
      src += ((size_t)(p.split ? wk.seg : sg.n) * p.H + head) * per_state + col;
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t] = ldg<f32x4>(src, lane_off + t * rows16);
    }
  }

  Stage<CH, DK, WK::THREADS> sx;
  Stage<CH, SSM_TILE, WK::THREADS> sy[SUBS];
  auto at = [&](int i) { return REV ? nch - 1 - i : i; };
  auto fetch = [&](int c) {
    const uint32_t tid = fresh(threadIdx.x);
    const int L = min(CH, sg.len - c * CH);
    sx.load_clamped(X + c * (CH * xp), 2 * (uint32_t)xp, L, tid);
#pragma unroll
    for (int i = 0; i < SUBS; ++i)
      sy[i].load_clamped(Y + c * (CH * yp) + (size_t)wk.head[i] * p.DV + wk.col[i], 2 * (uint32_t)yp, L, tid);
  };
  // wave i < TABS fills gate table i; the steps are loaded a chunk before they
  // are needed
  const int gh = TABS == 2 && w == 1 ? wk.head[SUBS - 1] : wk.head[0];
  const float A = p.A[gh], bias = p.bias ? p.bias[gh] : 0.f;
  double logd = 0.;
  auto load_dt = [&](int i) {
    const int c = at(min(i, nch - 1));
    return load_step(p, sg.row + (size_t)c * CH, min(CH, sg.len - c * CH), gh);
  };
  auto gates = [&](int i, float dt) {
    logd += fill_gates(lds.tabs[i & 1][w], dt + bias, A, min(CH, sg.len - at(i) * CH));
  };
  if (nch > 0) fetch(at(0));
  const int chunk0 = STORE ? first_chunk(p, sg) : 0;
  float sign = 1.f;  // of the accumulators
  float dt = 0.f;
  if (w < TABS && nch > 0) {
    gates(0, load_dt(0));
    dt = load_dt(1);
  }
  const uint32_t ax = lds_addr(lds.x), ay = lds_addr(lds.y);
  const typename XT::Col cx = XT::col_base(ax, l);
  const typename YT::Col cy = YT::col_base(ay, l);
  for (int i = 0; i < nch; ++i) {
    const int c = at(i);
    __syncthreads();
    const uint32_t tid = fresh(threadIdx.x);
    sx.template store_swz<DK>(ax, tid);
#pragma unroll
    for (int s = 0; s < SUBS; ++s) sy[s].template store_swz<YC>(ay, tid, s * SSM_TILE);
    __syncthreads();
    fetch(at(min(i + 1, nch - 1)));  // without a branch, which would hold two sets of registers
    const typename XT::Col bx = {fresh(cx.a), fresh(cx.b)};
    if (STORE) {
      float *dst = (REV ? p.dstates : p.states) + ((size_t)(chunk0 + c) * p.H + head) * per_state + col * DK;
#pragma unroll
      for (int t = 0; t < NT; ++t) stg<f32x4>(dst, chunk_state_unit<DK>(t, 0, m, g), sign * S[t]);
    }
    sign = -sign;
    const GateTab &T = lds.tabs[i & 1][TABS == 2 ? sub : 0];
    const float *coef = REV ? T.gam : T.ws;
    const float last = -T.last;
    Split ysp[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float y[8];
      unpack8(YT::col(cy, kb, w), y);
      const f32x4 c0 = sign * lds4(coef + 32 * kb + 8 * g), c1 = sign * lds4(coef + 32 * kb + 8 * g + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= e < 4 ? c0[e & 3] : c1[e & 3];
      ysp[kb] = split3(y);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 acc = S[t] * last;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 x = XT::col(bx, kb, t);
#pragma unroll
        for (int k = 2; k >= 0; --k) acc = mma32(acc, ysp[kb].p[k], x);
      }
      S[t] = acc;
    }
    if (w < TABS && i + 1 < nch) {
      gates(i + 1, dt);
      dt = load_dt(i + 2);
    }
  }
  // One writer an entry: the two directions run side by side and add the chunks in
  // opposite orders, so that the sums may differ in their last bit.  The reverse
  // sweep writes the last segment's, which the forward one skips.
  if (!STORE && w < TABS && l == 0 && wk.col[0] == 0 && (!REV || sg.last)) p.seg_decay[(size_t)wk.seg * p.H + gh] = logd;
  float *dst = nullptr;
  if (!STORE) dst = p.seg_state[REV] + ((size_t)wk.seg * p.H + head) * per_state;
  else if (REV && sg.first && p.dh0) dst = p.dh0 + ((size_t)sg.n * p.H + head) * per_state;
  if (!dst) return;
  mfma_settle();
#pragma unroll
  for (int t = 0; t < NT; ++t) stg<f32x4>(dst + col, lane_off + t * rows16, sign * S[t]);
}

// blockIdx.y: the forward sweep, or the reverse one
template <int DK, int PAIR, bool STORE>
__global__ __launch_bounds__(Work<PAIR>::THREADS, 4) void ssm_sweep_kernel(SsmParams p) {
  __shared__ SweepLds<DK, PAIR> lds;
  const int item = xcd_item(blockIdx.x, gridDim.x);
  if (blockIdx.y == 0)
    sweep<DK, PAIR, false, STORE>(p, lds, item);
  else
    sweep<DK, PAIR, true, STORE>(p, lds, item);
}

// ------------------------------------------------------------------- join
//
// Start states of a sequence's segments from their own end states and decays,
// in place, four state elements per thread; a sequence without tokens hands
// its initial state on.  Bound by the segment states' traffic, of which four
// segments are on their way at a time (32 segments of 32 heads of 128 x 64: 34
// MB read and written in 11 us, 6 TB/s; eight at a time take as long).
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
  constexpr int AHEAD = 4;
  for (int i = 0; i < cnt; i += AHEAD) {
    f32x4 *x[AHEAD], own[AHEAD];
    double d[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int j = min(i + k, cnt - 1);
      const size_t at = (size_t)(rev ? s0 + cnt - 1 - j : s0 + j) * p.H + h;
      x[k] = reinterpret_cast<f32x4 *>(st + at * per + e);
      if (i + k + 1 < cnt) {  // no sweep has filled the last one
        own[k] = *x[k];
        d[k] = p.seg_decay[at];
      } else {
        own[k] = zero4();
        d[k] = 0.;
      }
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (i + k >= cnt) break;
      *x[k] = cur;
      cur = cur * (float)exp2(d[k]) + own[k];
    }
  }
  float *out = rev ? p.dh0 : p.hT;
  if (cnt == 0 && out) *reinterpret_cast<f32x4 *>(out + (size_t)nh * per + e) = cur;
}

// ---------------------------------------------------------------- forward
//
// Per chunk: the lower 16 x 16 blocks of P = ((Q K^T) * Gamma) diag(s) (wave w
// computes row block w, rounded to bf16 into LDS; two heads share Q K^T), then
// every wave's columns of O^T = V^T P^T + diag(gamma) h^T Q^T and of the state
// update.  Two stacked state tiles (rows Dk, columns the wave's 16) are the
// operand of h^T Q^T as they stand.  While the other waves compute P, waves 0
// and 1, whose row blocks are the shortest, fill the next chunk's gate tables.
//
// Bound by issue: a chunk of two heads costs a wave 150 products, 96 of them the
// state update in three parts, and some 900 vector instructions, and the two
// kinds share a SIMD's turns (77 % of the cycles; twice the waves of half the
// work each spill).  4 x 4096 tokens, 32 heads of 128 x 64: 71 us.
template <int DK, int PAIR>
struct FwdLds {
  static constexpr int VC = SSM_TILE * Work<PAIR>::SUBS;
  alignas(256) bf16 q[CH * DK];
  alignas(256) bf16 k[CH * DK];
  alignas(256) bf16 v[CH * VC];
  alignas(256) bf16 p[Work<PAIR>::TABS][CH * CH];
  GateTab tabs[2][Work<PAIR>::TABS];
};

template <int DK, int PAIR>
__global__ __launch_bounds__(NTHR, 2) void ssm_fwd_kernel(SsmParams p) {
  using WK = Work<PAIR>;
  using QT = Swz<DK>;
  using VT = Swz<FwdLds<DK, PAIR>::VC>;
  using PT = Swz<CH>;
  constexpr int MT = DK / 16, KB = DK / 32, SUBS = WK::SUBS, TABS = WK::TABS, VC = FwdLds<DK, PAIR>::VC;
  __shared__ FwdLds<DK, PAIR> lds;
  if (p.zero_tail) clear_tail<u32x4>(p, p.o, (int64_t)p.H * p.DV / 8);
  const WK wk(p, xcd_item(blockIdx.x, gridDim.x));
  Segment sg;
  if (!segment(p, wk.seg, sg)) return;
  const int w = wave_number(), l = lane_id(), g = l >> 4, m = l & 15;
  const int grp = wk.head[0] / (p.H / p.G);
  const size_t kp = (size_t)p.G * DK, vp = (size_t)p.H * p.DV;
  const bf16 *Q = p.q + sg.row * kp + (size_t)grp * DK, *K = p.k + sg.row * kp + (size_t)grp * DK;
  const int nch = (sg.len + CH - 1) / CH;
  const size_t per_state = (size_t)DK * p.DV;
  size_t vo[SUBS];  // the half's first token and column
  float skip[SUBS];
#pragma unroll
  for (int s = 0; s < SUBS; ++s) {
    vo[s] = sg.row * vp + (size_t)wk.head[s] * p.DV + wk.col[s];
    skip[s] = p.skip ? p.skip[wk.head[s]] : 0.f;
  }

  f32x4 S[SUBS][MT];  // rows 16 t + 4 g + i, column m of the wave's 16 in each half
#pragma unroll
  for (int s = 0; s < SUBS; ++s) {
    const float *src = p.split ? p.seg_state[0] : p.h0;
    if (src) src += ((size_t)(p.split ? wk.seg : sg.n) * p.H + wk.head[s]) * per_state + wk.col[s] + 16 * w;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[s][t][i] = src ? ldg<float>(src, 4 * ((16 * t + 4 * g + i) * p.DV + m)) : 0.f;
  }

  Stage<CH, DK, NTHR> sq, sk;
  Stage<CH, SSM_TILE, NTHR> sv[SUBS];
  auto fetch = [&](int c) {
    const uint32_t tid = fresh(threadIdx.x);
    const int L = min(CH, sg.len - c * CH);
    sq.load_clamped(Q + c * (CH * kp), 2 * (uint32_t)kp, L, tid);
    sk.load_clamped(K + c * (CH * kp), 2 * (uint32_t)kp, L, tid);
#pragma unroll
    for (int s = 0; s < SUBS; ++s) sv[s].load_clamped(p.v + vo[s] + c * (CH * vp), 2 * (uint32_t)vp, L, tid);
  };
  // wave i < TABS, which has the least of P to compute, fills gate table i; the
  // steps are loaded a chunk before they are needed
  const int gh = TABS == 2 && w == 1 ? wk.head[SUBS - 1] : wk.head[0];
  const float A = p.A[gh], bias = p.bias ? p.bias[gh] : 0.f;
  auto load_dt = [&](int i) {
    const int c = min(i, nch - 1);
    return load_step(p, sg.row + (size_t)c * CH, min(CH, sg.len - c * CH), gh);
  };
  auto gates = [&](int c, float dt) { fill_gates(lds.tabs[c & 1][w], dt + bias, A, min(CH, sg.len - c * CH)); };
  if (nch > 0) fetch(0);
  float dt = 0.f;
  if (w < TABS && nch > 0) {
    gates(0, load_dt(0));
    dt = load_dt(1);
  }
  const uint32_t aq = lds_addr(lds.q), ak = lds_addr(lds.k), av = lds_addr(lds.v), ap = lds_addr(lds.p);
  // the block right of an even diagonal block stays zero
  if (w % 2 == 0)
#pragma unroll
    for (int t = 0; t < TABS; ++t) wy::st(PT::quad(PT::quad_base(ap, l), w, w + 1) + t * (2 * CH * CH), cvt_bf16x4(zero4()));
  for (int c = 0; c < nch; ++c) {
    const int L = min(CH, sg.len - c * CH);
    __syncthreads();
    {
      const uint32_t tid = fresh(threadIdx.x);
      sq.template store_swz<DK>(aq, tid);
      sk.template store_swz<DK>(ak, tid);
#pragma unroll
      for (int s = 0; s < SUBS; ++s) sv[s].template store_swz<VC>(av, tid, s * SSM_TILE);
    }
    __syncthreads();
    fetch(min(c + 1, nch - 1));  // without a branch, which would hold two sets of registers
    const int l = fresh(lane_id()), g = l >> 4, m = l & 15;

    // P, row block w: tiles hold rows j (four per lane), column r
    {
      const uint32_t rq = QT::row_base(aq, l), rk = rq + (ak - aq), pq = PT::quad_base(ap, l);
      const int r = 16 * w + m;
      bf16x8 qf[KB];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) qf[kb] = QT::row(rq, w, kb);
      for (int jb = 0; jb <= w; ++jb) {
        const int j0 = 16 * jb + 4 * g;
        f32x4 acc = zero4();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) acc = mma32(acc, QT::row(rk, jb, kb), qf[kb]);
#pragma unroll
        for (int t = 0; t < TABS; ++t) {
          const GateTab &T = lds.tabs[c & 1][t];
          const f32x4 gm = decay_ratios(T, j0, T.bh[r], T.bl[r], -1.f), sj = lds4(T.s + j0);
          f32x4 pr;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = computed(acc[i] * (gm[i] * sj[i]));
            pr[i] = j0 + i <= r ? x : 0.f;
          }
          wy::st(PT::quad(pq, w, jb) + t * (2 * CH * CH), cvt_bf16x4(pr));
        }
      }
    }
    if (w < TABS && c + 1 < nch) {
      gates(c + 1, dt);
      dt = load_dt(c + 2);
    }
    __syncthreads();

    // O^T tiles: rows the wave's 16 columns, column r
    bf16x8 vf[SUBS][2];
    {
      const typename VT::Col cv = VT::col_base(av, l);
#pragma unroll
      for (int s = 0; s < SUBS; ++s)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) vf[s][kb] = VT::col(cv, kb, 4 * s + w);
    }
    {
      const uint32_t qq = QT::quad_base(aq, l), vq = VT::quad_base(av, l), rp = PT::row_base(ap, l);
      const uint32_t row_off = 2 * (m * (uint32_t)vp + 16 * w + 4 * g);
      bf16x8 sf[SUBS][KB];
#pragma unroll
      for (int s = 0; s < SUBS; ++s)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) sf[s][kb] = bfrag<bf16>(S[s][2 * kb], S[s][2 * kb + 1]);
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) {
        const int r = 16 * rb + m;
        f32x4 a[SUBS], b[SUBS];
#pragma unroll
        for (int s = 0; s < SUBS; ++s) a[s] = b[s] = zero4();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const bf16x8 qf = QT::row_stacked(qq, rb, kb);
#pragma unroll
          for (int s = 0; s < SUBS; ++s) b[s] = mma32(b[s], sf[s][kb], qf);
        }
#pragma unroll
        for (int kb = 0; kb <= rb / 2; ++kb)
#pragma unroll
          for (int s = 0; s < SUBS; ++s)
            a[s] = mma32(a[s], vf[s][kb], PT::row(rp + (TABS == 2 ? s : 0) * (2 * CH * CH), rb, kb));
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
          const bf16x4 vr = wy::ld<bf16x4>(VT::quad(vq ^ (32 * w), rb, 4 * s));
          const float gam = lds.tabs[c & 1][TABS == 2 ? s : 0].gam[r];
          f32x4 o;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = a[s][i] + gam * b[s][i] + skip[s] * (float)vr[i];
          if (r < L) stg<bf16x4>(p.o + vo[s] + c * (CH * vp) + rb * (16 * vp), row_off, cvt_bf16x4(o));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // state update
    const typename QT::Col ck = QT::col_base(ak, l);
    Split vsp[SUBS][2];
#pragma unroll
    for (int s = 0; s < SUBS; ++s) {
      const GateTab &T = lds.tabs[c & 1][TABS == 2 ? s : 0];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        float x[8];
        unpack8(vf[s][kb], x);
        const f32x4 c0 = lds4(T.ws + 32 * kb + 8 * g), c1 = lds4(T.ws + 32 * kb + 8 * g + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= e < 4 ? c0[e & 3] : c1[e & 3];
        vsp[s][kb] = split3(x);
      }
      const float last = T.last;
#pragma unroll
      for (int t = 0; t < MT; ++t) S[s][t] *= last;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 kf = QT::col(ck, kb, t);
#pragma unroll
        for (int k = 2; k >= 0; --k)
#pragma unroll
          for (int s = 0; s < SUBS; ++s) S[s][t] = mma32(S[s][t], kf, vsp[s][kb].p[k]);
      }
    }
  }
  if (p.hT && sg.last) {
    mfma_settle();
#pragma unroll
    for (int s = 0; s < SUBS; ++s) {
      float *dst = p.hT + ((size_t)sg.n * p.H + wk.head[s]) * per_state + wk.col[s] + 16 * w;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) stg<float>(dst, 4 * ((16 * t + 4 * g + i) * p.DV + m), S[s][t][i]);
    }
  }
}

template <int DK, int PAIR>
void start_sweep(const SsmParams &p, bool store, const dim3 &grid, hipStream_t stream) {
  if (store) hipLaunchKernelGGL((ssm_sweep_kernel<DK, PAIR, true>), grid, dim3(Work<PAIR>::THREADS), 0, stream, p);
  else hipLaunchKernelGGL((ssm_sweep_kernel<DK, PAIR, false>), grid, dim3(Work<PAIR>::THREADS), 0, stream, p);
}

}  // namespace

hipError_t launch_ssm_sweep(const SsmParams &p, int DK, bool store, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)work_items(p), backward ? 2 : 1);
  if (grid.x == 0) return hipSuccess;
  if (DK == 64) {
    if (p.pair == SSM_TILES) start_sweep<64, SSM_TILES>(p, store, grid, stream);
    else if (p.pair == SSM_HEADS) start_sweep<64, SSM_HEADS>(p, store, grid, stream);
    else start_sweep<64, SSM_SINGLE>(p, store, grid, stream);
  } else {
    if (p.pair == SSM_TILES) start_sweep<128, SSM_TILES>(p, store, grid, stream);
    else if (p.pair == SSM_HEADS) start_sweep<128, SSM_HEADS>(p, store, grid, stream);
    else start_sweep<128, SSM_SINGLE>(p, store, grid, stream);
  }
  return hipGetLastError();
}

hipError_t launch_ssm_join(const SsmParams &p, int DK, bool backward, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.N * p.H * DK * p.DV / (4 * JOIN_THREADS)), backward ? 2 : 1);
  hipLaunchKernelGGL(ssm_join_kernel, grid, dim3(JOIN_THREADS), 0, stream, p, DK);
  return hipGetLastError();
}

template <int DK>
static void start_fwd(const SsmParams &p, unsigned grid, hipStream_t stream) {
  if (p.pair == SSM_TILES) hipLaunchKernelGGL((ssm_fwd_kernel<DK, SSM_TILES>), dim3(grid), dim3(NTHR), 0, stream, p);
  else if (p.pair == SSM_HEADS) hipLaunchKernelGGL((ssm_fwd_kernel<DK, SSM_HEADS>), dim3(grid), dim3(NTHR), 0, stream, p);
  else hipLaunchKernelGGL((ssm_fwd_kernel<DK, SSM_SINGLE>), dim3(grid), dim3(NTHR), 0, stream, p);
}

hipError_t launch_ssm_fwd(const SsmParams &p, int DK, hipStream_t stream) {
  const unsigned grid = (unsigned)work_items(p);
  if (grid == 0) return hipSuccess;
  if (DK == 64) start_fwd<64>(p, grid, stream);
  else start_fwd<128>(p, grid, stream);
  return hipGetLastError();
}

}  // namespace dn
