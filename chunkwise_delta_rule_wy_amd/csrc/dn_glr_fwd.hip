// Gated linear recurrence, forward pass, segment maps of both directions, and
// the single-token step (dn_glr.h has the mathematics).
//
// Uncut, the forward pass is bound by memory and near its vector instructions, which
// keep the units busy in 61 % of the cycles: 4 x 4096 tokens of 4096 channels in bf16 120 us,
// 4.5 TB/s.  A thread's run of eight rows, whose maps it composes and then walks again with
// their gates still in registers, is loaded a tile ahead.  The segments' maps (16384
// tokens of 2048 channels: 46 us, 4.4 TB/s) are bound by vector instructions; there loads
// ahead of the arithmetic gained nothing.
#include "dn_glr.h"

namespace dn {
namespace {

constexpr int ROWS = GLR_TILE / GLR_RUNS;  // rows of a run

// The maps of the first `count` of every NS segments (going back the last): a thread
// walks through one sixteenth of its segment's rows, and the runs' maps meet in LDS at
// the end.
template <typename E, bool BACK>
__global__ __launch_bounds__(GLR_THREADS) void glr_sum_kernel(GlrParams p, int count) {
  typedef typename Pair<E>::type P2;
  __shared__ f32x4 maps[GLR_RUNS][GLR_LANES];
  const int nth = blockIdx.x / p.groups, grp = blockIdx.x % p.groups;
  const int seg = nth / count * p.NS + nth % count + (BACK ? p.NS - count : 0);
  const int lane = threadIdx.x % GLR_LANES, run = threadIdx.x / GLR_LANES;
  const int ch = grp * GLR_CH + 2 * lane, c = min(ch, p.C - 2);
  const GlrSegment s = glr_segment(p, seg);
  const GlrChannel k0 = glr_channel(p.lam, p.br, p.bi, p.power, c), k1 = glr_channel(p.lam, p.br, p.bi, p.power, c + 1);
  const int per = p.segt * (GLR_TILE / GLR_RUNS);  // rows of a run, a multiple of ROWS
  const int64_t beg = s.row0 + (int64_t)run * per, end = min(beg + per, s.row1);
  f32x2 A = {1.f, 1.f}, B = {0.f, 0.f};
  bool closed = false;  // going back: the rows from here on are behind a sequence's end
  // the sequences of the first rows of the wave's two runs
  GlrSeq q, upper;
  const int64_t first = s.row0 + (int64_t)__builtin_amdgcn_readfirstlane(2 * wave_id()) * per;
  q.find(p, min(first, s.row1 - 1));
  upper.find(p, min(first + per, s.row1 - 1));
  if (run & 1) q = upper;
  // in row order: going back the maps are composed on the other side, c -> A (a c + b) + B
  for (int64_t row = beg; row < end; row += ROWS) {
    P2 r[ROWS], x[ROWS], i[ROWS];
    const int left = (int)min(end - row, (int64_t)ROWS);
    glr_load_at<E>(p.r, row, left, p.C, c, r);
    glr_load_at<E>(BACK ? p.dy : p.x, row, left, p.C, c, x);
    if (!BACK) glr_load_at<E>(p.i, row, left, p.C, c, i);
    f32x2 a[ROWS], b[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const f32x2 rj = to_f2<E>(r[j]), xj = to_f2<E>(x[j]);
      const float l0 = k0.k2 * glr_sigmoid(rj[0], k0.br), l1 = k1.k2 * glr_sigmoid(rj[1], k1.br);
      a[j] = (f32x2){__builtin_amdgcn_exp2f(l0), __builtin_amdgcn_exp2f(l1)};
      if (BACK) {
        b[j] = (f32x2){a[j][0] * xj[0], a[j][1] * xj[1]};
      } else {
        const f32x2 ij = to_f2<E>(i[j]);
        b[j] = (f32x2){__builtin_amdgcn_sqrtf(glr_rest(a[j][0], l0)) * glr_sigmoid(ij[0], k0.bi) * xj[0],
                       __builtin_amdgcn_sqrtf(glr_rest(a[j][1], l1)) * glr_sigmoid(ij[1], k1.bi) * xj[1]};
      }
    }
    GlrFlags f;
    if (__any(glr_flags<ROWS>(p, q, row, end, f))) {
      GlrSeq w = q;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        if (j >= f.live) {
          a[j] = (f32x2){1.f, 1.f};
          b[j] = (f32x2){0.f, 0.f};
        } else if (f.dead >> j & 1) {
          a[j] = (f32x2){GLR_CUT, GLR_CUT};
          b[j] = (f32x2){0.f, 0.f};
        } else if ((BACK ? f.ends : f.starts) >> j & 1) {
          // the state in front of the row, or the gradient behind it, is h0 or dhT
          w.walk(p, row + j);
          const float *st = BACK ? p.dhT : p.h0;
          if (st) b[j] = glr_fma(a[j], *reinterpret_cast<const f32x2 *>(st + (size_t)w.n * p.C + c), b[j]);
          a[j] = (f32x2){GLR_CUT, GLR_CUT};
        }
        B = BACK ? glr_map(A, b[j], B) : glr_map(a[j], B, b[j]);
        A = glr_times(A, a[j]);
      }
      closed |= (f.dead | f.ends) != 0;
    } else if (!BACK || !closed) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        B = BACK ? glr_fma(A, b[j], B) : glr_fma(a[j], B, b[j]);
        A = (f32x2){A[0] * a[j][0], A[1] * a[j][1]};
      }
    }
  }
  maps[run][lane] = (f32x4){A[0], A[1], B[0], B[1]};
  __syncthreads();
  if (threadIdx.x >= GLR_LANES || ch >= p.C) return;
  A = (f32x2){1.f, 1.f};
  B = (f32x2){0.f, 0.f};
#pragma unroll
  for (int k = 0; k < GLR_RUNS; ++k) {
    const f32x4 m = maps[BACK ? GLR_RUNS - 1 - k : k][lane];
    A = glr_times(A, (f32x2){m[0], m[1]});
    B = glr_map((f32x2){m[0], m[1]}, B, (f32x2){m[2], m[3]});
  }
  float *out = (BACK ? p.sum_r : p.sum_f) + (size_t)seg * 2 * p.C + ch;
  *reinterpret_cast<f32x2 *>(out) = A;
  *reinterpret_cast<f32x2 *>(out + p.C) = B;
}

template <typename E, bool FLAT, bool Y>
__global__ __launch_bounds__(GLR_THREADS) void glr_fwd_kernel(GlrParams p) {
  typedef typename Pair<E>::type P2;
  __shared__ f32x4 maps[2][GLR_WAVES][GLR_LANES];
  const int seg = blockIdx.x / p.groups, grp = blockIdx.x % p.groups;
  const int lane = threadIdx.x % GLR_LANES, run = threadIdx.x / GLR_LANES, wave = wave_id();
  // lanes behind the last channels repeat them, stores included
  const int c = min(grp * GLR_CH + 2 * lane, p.C - 2);
  const GlrSegment s = glr_segment(p, seg);
  const GlrChannel k0 = glr_channel(p.lam, p.br, p.bi, p.power, c), k1 = glr_channel(p.lam, p.br, p.bi, p.power, c + 1);
  // sequences without tokens pass h0 on
  if (p.hT && (p.cu || p.T == 0))
    for (int64_t n = (int64_t)seg * GLR_RUNS + run; n < p.N; n += (int64_t)p.nseg * GLR_RUNS)
      if (!p.cu || p.cu[n] == p.cu[n + 1])
        *reinterpret_cast<f32x2 *>(p.hT + n * p.C + c) =
            p.h0 ? *reinterpret_cast<const f32x2 *>(p.h0 + n * p.C + c) : (f32x2){0.f, 0.f};
  f32x2 carry = {0.f, 0.f};  // the state in front of the tile
  GlrSeq q;
  const int first = glr_reach<false>(p, s, seg, q);
  if (p.cut) carry = glr_join<false>(p, p.sum_f, first, seg, c, &maps[0][0][0]);
  if (s.row0 >= s.row1) return;
  P2 x[ROWS], r[ROWS], i[ROWS];
  // No branch in the loads: registers that are loaded in one of two ways get copied
  // where these meet, and the copies wait.
  const uint32_t pitch = p.C * (uint32_t)sizeof(E), col = c * (uint32_t)sizeof(E);
  const auto load = [&](int64_t tile) {
    uint32_t o[ROWS];
    glr_offsets<ROWS>(o, run * ROWS, (int)min(s.row1 - tile, (int64_t)GLR_TILE), pitch, col);
    glr_load<E>(p.x, tile, o, p.C, x);
    glr_load<E>(p.r, tile, o, p.C, r);
    glr_load<E>(p.i, tile, o, p.C, i);
  };
  load(s.row0);
  glr_settle();
  int turn = 0;
  int64_t block = s.state0;
  for (int64_t tile = s.row0; tile < s.row1; tile += GLR_TILE, turn ^= 1, block += GLR_TILE / GLR_STATE) {
    const int64_t row = tile + run * ROWS;
    GlrFlags f = {0, 0, 0, ROWS};
    // in a segment of one sequence only its outer tiles have rows that need care
    const bool slow = (FLAT || tile == s.row0 || tile + GLR_TILE >= s.row1) && __any(glr_flags<ROWS>(p, q, row, s.row1, f));
    f32x2 a[ROWS], b[ROWS], A = {1.f, 1.f}, B = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const f32x2 xj = to_f2<E>(x[j]), rj = to_f2<E>(r[j]), ij = to_f2<E>(i[j]);
      const float l0 = k0.k2 * glr_sigmoid(rj[0], k0.br), l1 = k1.k2 * glr_sigmoid(rj[1], k1.br);
      a[j] = (f32x2){__builtin_amdgcn_exp2f(l0), __builtin_amdgcn_exp2f(l1)};
      b[j] = (f32x2){__builtin_amdgcn_sqrtf(glr_rest(a[j][0], l0)) * glr_sigmoid(ij[0], k0.bi) * xj[0],
                     __builtin_amdgcn_sqrtf(glr_rest(a[j][1], l1)) * glr_sigmoid(ij[1], k1.bi) * xj[1]};
    }
    load(tile + GLR_TILE < s.row1 ? tile + GLR_TILE : s.row0);  // behind the last one the first again
    if (slow) {
      GlrSeq w = q;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        if (j >= f.live) {
          a[j] = (f32x2){1.f, 1.f};
          b[j] = (f32x2){0.f, 0.f};
        } else if (f.dead >> j & 1) {
          a[j] = (f32x2){GLR_CUT, GLR_CUT};
          b[j] = (f32x2){0.f, 0.f};
        } else if (f.starts >> j & 1) {
          w.walk(p, row + j);
          if (p.h0) b[j] = glr_fma(a[j], *reinterpret_cast<const f32x2 *>(p.h0 + (size_t)w.n * p.C + c), b[j]);
          a[j] = (f32x2){GLR_CUT, GLR_CUT};
        }
        B = glr_map(a[j], B, b[j]);
        A = glr_times(A, a[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        B = glr_fma(a[j], B, b[j]);
        A = (f32x2){A[0] * a[j][0], A[1] * a[j][1]};
      }
    }
    // a wave's two runs, then the waves
    const f32x2 oA = other_half(A), oB = other_half(B);
    const bool upper = threadIdx.x & 32;
    if (!upper) {
      const f32x2 tB = glr_map<FLAT>(oA, B, oB);
      const f32x2 tA = glr_times<FLAT>(A, oA);
      maps[turn][wave][lane] = (f32x4){tA[0], tA[1], tB[0], tB[1]};
    }
    __syncthreads();
    f32x2 h = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < GLR_WAVES; ++k) {
      if (k == wave) h = carry;
      if (p.states && k % (GLR_WAVES * GLR_STATE / GLR_TILE) == 0 && k == wave && !upper &&
          tile + k * (GLR_TILE / GLR_WAVES) < s.row1)
        *reinterpret_cast<f32x2 *>(p.states + (block + k / (GLR_WAVES * GLR_STATE / GLR_TILE)) * p.C + c) = carry;
      const f32x4 m = maps[turn][k][lane];
      carry = glr_map<FLAT>((f32x2){m[0], m[1]}, carry, (f32x2){m[2], m[3]});
    }
    if (upper) h = glr_map<FLAT>(oA, h, oB);
    uint32_t o[ROWS];
    glr_offsets<ROWS>(o, run * ROWS, GLR_TILE, pitch, col);
    if (slow) {
      GlrSeq w = q;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        h = glr_map(a[j], h, b[j]);
        if (j < f.live) {
          if (Y && (!(f.dead >> j & 1) || p.zero_tail)) glr_store(glr_base(p.y, tile * pitch), o[j], to_e2<E>(h));
          if (p.hT && f.ends >> j & 1) {
            w.walk(p, row + j);
            *reinterpret_cast<f32x2 *>(p.hT + (size_t)w.n * p.C + c) = h;
          }
        }
      }
      glr_settle();
    } else {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        h = glr_fma(a[j], h, b[j]);
        if (Y) glr_store(glr_base(p.y, tile * pitch), o[j], to_e2<E>(h));
      }
    }
  }
}

// One token: a thread takes four channels of ROWS sequences, whose gates' constants
// it computes once.
constexpr int STEP_THREADS = 256;

template <typename E, int ROWS>
__global__ __launch_bounds__(STEP_THREADS) void glr_step_kernel(GlrStepParams p) {
  typedef typename four<E>::type E4;
  const int c = (blockIdx.x * STEP_THREADS + threadIdx.x) * 4, b0 = blockIdx.y * ROWS;
  if (c >= p.C) return;
  E4 x[ROWS], r[ROWS], i[ROWS];
  f32x4 h[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const size_t at = (size_t)min(b0 + j, p.B - 1) * p.C + c;
    x[j] = *reinterpret_cast<const E4 *>(static_cast<const E *>(p.x) + at);
    r[j] = *reinterpret_cast<const E4 *>(static_cast<const E *>(p.r) + at);
    i[j] = *reinterpret_cast<const E4 *>(static_cast<const E *>(p.i) + at);
    h[j] = *reinterpret_cast<const f32x4 *>(p.state + at);
  }
  GlrChannel k[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) k[e] = glr_channel(p.lam, p.br, p.bi, p.power, c + e);
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if (b0 + j >= p.B) break;
    const size_t at = (size_t)(b0 + j) * p.C + c;
    E4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float l2 = k[e].k2 * glr_sigmoid(to_f<E>(r[j][e]), k[e].br), a = __builtin_amdgcn_exp2f(l2);
      const float u = glr_sigmoid(to_f<E>(i[j][e]), k[e].bi) * to_f<E>(x[j][e]);
      h[j][e] = __builtin_fmaf(a, h[j][e], __builtin_amdgcn_sqrtf(glr_rest(a, l2)) * u);
      y[e] = to_e<E>(h[j][e]);
    }
    *reinterpret_cast<f32x4 *>(p.state + at) = h[j];
    *reinterpret_cast<E4 *>(static_cast<E *>(p.y) + at) = y;
  }
}

}  // namespace

// Nothing follows a sequence's last segment (going back its first), whose map is left
// out, except where all that the forward pass reads stays in the last cache of 256 MB:
// there that segment would be the only one that is read from memory in the pass after
// (16384 rows in bf16, forwards, without it [with it]: 2048 channels 108 us [104], 4096 in
// packed sequences 206 [215]; backwards 141 [145] and 270 [282]).
hipError_t launch_glr_sum(const GlrParams &p, int dtype, bool backward, hipStream_t st) {
  const int64_t bytes = 3 * p.rows * p.C * (dtype == 1 ? 2 : 4);
  const int count = !backward && bytes <= 256 << 20 ? p.NS : p.NS - 1;
  const dim3 grid((unsigned)((int64_t)(p.nseg / p.NS) * count * p.groups)), thr(GLR_THREADS);
  if (dtype == 1) {
    if (backward) hipLaunchKernelGGL((glr_sum_kernel<bf16, true>), grid, thr, 0, st, p, count);
    else hipLaunchKernelGGL((glr_sum_kernel<bf16, false>), grid, thr, 0, st, p, count);
  } else {
    if (backward) hipLaunchKernelGGL((glr_sum_kernel<float, true>), grid, thr, 0, st, p, count);
    else hipLaunchKernelGGL((glr_sum_kernel<float, false>), grid, thr, 0, st, p, count);
  }
  return hipGetLastError();
}

hipError_t launch_glr_fwd(const GlrParams &p, int dtype, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.nseg * p.groups)), thr(GLR_THREADS);
  const auto go = [&](auto e, auto y) {
    typedef decltype(e) E;
    constexpr bool Y = decltype(y)::value;
    if (p.flat) hipLaunchKernelGGL((glr_fwd_kernel<E, true, Y>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((glr_fwd_kernel<E, false, Y>), grid, thr, 0, st, p);
  };
  if (dtype == 1) p.y ? go(bf16(), std::true_type()) : go(bf16(), std::false_type());
  else p.y ? go(0.f, std::true_type()) : go(0.f, std::false_type());
  return hipGetLastError();
}

// Four sequences a thread where single ones would give the CUs two workgroups and more
// (4096 channels in bf16, 256 sequences: 6.0 us, single 8.2, eight 7.2; 64 sequences: 5.0 us,
// single 4.1).
hipError_t launch_glr_step(const GlrStepParams &p, int dtype, hipStream_t st) {
  const int64_t cols = (p.C / 4 + STEP_THREADS - 1) / STEP_THREADS;
  const bool many = cols * p.B >= 512;
  const dim3 grid((unsigned)cols, (unsigned)(many ? (p.B + 3) / 4 : p.B)), thr(STEP_THREADS);
  if (dtype == 1) {
    if (many) hipLaunchKernelGGL((glr_step_kernel<bf16, 4>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((glr_step_kernel<bf16, 1>), grid, thr, 0, st, p);
  } else {
    if (many) hipLaunchKernelGGL((glr_step_kernel<float, 4>), grid, thr, 0, st, p);
    else hipLaunchKernelGGL((glr_step_kernel<float, 1>), grid, thr, 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace dn
