// Depthwise causal short convolution with bias, SiLU and a carried state, its
// backward and its single-token step, for gfx950.  Per channel c of C = H D,
// inside one sequence whose inputs before the first token are the carried
// state s0 (its last W - 1 inputs; zeros without one):
//
//   z[t] = bias + sum_{j < W} w[j] x[t - (W - 1) + j],   y[t] = z[t] sigmoid(z[t])
//   sT   = the last W - 1 inputs
//   dz   = dy sigmoid(z) (1 + z (1 - sigmoid(z)))
//   dx[p] = sum_j w[j] dz[p + (W - 1) - j] (+ dsT), the same for the places before
//           the first token, which are ds0
//   dw[j] = sum_t dz[t] x[t - (W - 1) + j],  dbias = sum_t dz[t]
//
// A thread owns four consecutive channels (8 bytes of bf16, 16 of fp32) of a
// run of consecutive tokens and slides the W-token window through registers; a
// run reads the W - 1 rows beside it again.  Everything else is streamed once:
// HBM bounds the forward pass and the step, HBM and some 35 vector instructions
// an element the backward pass, in which a thread recomputes z from x.  Rows are
// loaded in batches, in the backward pass a batch ahead of their use.  Measured
// at 4 x 4096 tokens of 4096 channels, W = 4, bf16: 53 us forwards (5.1 TB/s,
// the rate of a large copy; with eight channels and eight rows 55 us) and 90 us
// backwards (4.5 TB/s; batches of one row 93 us, of four, which leave three waves
// on a SIMD, 97 us, of four without the early loads 93 us).  In fp32 both passes
// together, whole calls, take 267 us: 1.34 GB at 5.0 TB/s.  The weights' gradients
// are summed in registers over a run, in LDS over a workgroup's runs and by a
// second kernel over the workgroups, in a fixed order, so that they repeat bit for
// bit.
#include "dn.h"
#include "dn_rows.h"

namespace dn {
namespace {

constexpr int CS_THREADS = 256;
constexpr int CS_CH = 4;         // channels of a thread
constexpr int CS_BATCH = 4;      // rows loaded ahead (forward)
constexpr int CS_BWD_BATCH = 2;  // the same of x and dy, a batch ahead of their use
constexpr int CS_MAX_ROWS = 256; // rows of partial weight gradients

struct ConvSiluParams {
  const void *x, *s0, *dy, *dsT;  // s0, dsT may be null
  const float *w, *bias;          // bias may be null
  const int32_t *cu;
  void *y, *sT, *dx, *ds0;        // sT, ds0 may be null
  float *part, *dw, *dbias;       // part [rows][C][W + 1]; dbias may be null
  int64_t TT;
  int T, N, C, W, run;
  int runs, rows;
  int zero_tail;  // packed: clear the rows of y or dx behind the last sequence
};

// a row's CS_CH channels as they are in memory
template <typename E>
struct Raw {
  typedef E V __attribute__((ext_vector_type(CS_CH)));
  V v;
  __device__ __forceinline__ void load(const E *src, bool valid) {
    if (valid) v = *reinterpret_cast<const V *>(src);
    else
#pragma unroll
      for (int e = 0; e < CS_CH; ++e) v[e] = to_e<E>(0.f);
  }
  __device__ __forceinline__ void get(float (&x)[CS_CH]) const {
#pragma unroll
    for (int e = 0; e < CS_CH; ++e) x[e] = to_f<E>(v[e]);
  }
};

template <typename E>
__device__ __forceinline__ void load_ch(const E *src, float (&x)[CS_CH]) {
  Raw<E> r;
  r.load(src, true);
  r.get(x);
}
template <typename E>
__device__ __forceinline__ void store_ch(E *dst, const float (&x)[CS_CH]) {
  typedef E V __attribute__((ext_vector_type(CS_CH)));
  V v;
#pragma unroll
  for (int e = 0; e < CS_CH; ++e) v[e] = to_e<E>(x[e]);
  *reinterpret_cast<V *>(dst) = v;
}
// a thread's channels of those of a result's rows [t, end) that are behind the
// last sequence; called before a run holds anything in registers (behind its
// loop the backward pass spills)
template <typename E>
__device__ __forceinline__ void clear_tail(const ConvSiluParams &p, void *result, int64_t t, int64_t end, int c0) {
  if (!p.zero_tail) return;
  typedef E V __attribute__((ext_vector_type(CS_CH)));
  for (t = max(t, (int64_t)p.cu[p.N]); t < end; ++t) *reinterpret_cast<V *>(static_cast<E *>(result) + t * p.C + c0) = V{};
}
__device__ __forceinline__ void zero_ch(float (&x)[CS_CH]) {
#pragma unroll
  for (int e = 0; e < CS_CH; ++e) x[e] = 0.f;
}
// the sequence [st, nx) around token t, number n
struct Seq {
  int n;
  int64_t st, nx;
  __device__ __forceinline__ void find(const ConvSiluParams &p, int64_t t) {
    if (!p.cu) {
      n = (int)(t / p.T);
      st = (int64_t)n * p.T;
      nx = st + p.T;
      return;
    }
    int lo = 0, hi = p.N - 1;  // the last n with cu[n] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    n = lo;
    st = p.cu[n];
    nx = p.cu[n + 1];
  }
};

// the thread's W x CS_CH weights lie together; w and bias are 16-byte aligned
template <int W>
__device__ __forceinline__ void load_weights(const float *wt, const float *bias, int c0, float (&w)[W][CS_CH],
                                             float (&b)[CS_CH]) {
  float f[W * CS_CH];
  load_f32<W * CS_CH>(wt + (size_t)c0 * W, f);
#pragma unroll
  for (int e = 0; e < CS_CH; ++e)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
  if (bias) load_f32<CS_CH>(bias + c0, b);
  else zero_ch(b);
}

// the W - 1 inputs before token t of sequence s
template <typename E, int W>
__device__ __forceinline__ void load_history(const ConvSiluParams &p, const Seq &s, int64_t t, int c0,
                                             float (&h)[W > 1 ? W - 1 : 1][CS_CH]) {
  const E *x = static_cast<const E *>(p.x), *s0 = static_cast<const E *>(p.s0);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int64_t i = t - (W - 1) + k;
    if (i >= s.st) load_ch<E>(x + i * p.C + c0, h[k]);
    else if (s0) load_ch<E>(s0 + ((int64_t)s.n * (W - 1) + (i - s.st) + (W - 1)) * p.C + c0, h[k]);
    else zero_ch(h[k]);
  }
}
template <int N>
__device__ __forceinline__ void shift(float (&h)[N][CS_CH], const float (&x)[CS_CH]) {
#pragma unroll
  for (int k = 0; k + 1 < N; ++k)
#pragma unroll
    for (int e = 0; e < CS_CH; ++e) h[k][e] = h[k + 1][e];
#pragma unroll
  for (int e = 0; e < CS_CH; ++e) h[N - 1][e] = x[e];
}
__device__ __forceinline__ float sigmoidf(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

template <int W>
__device__ __forceinline__ float conv_at(const float (&w)[W][CS_CH], const float (&b)[CS_CH],
                                         const float (&h)[W > 1 ? W - 1 : 1][CS_CH], const float (&x)[CS_CH], int e) {
  float z = b[e] + w[W - 1][e] * x[e];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) z += w[j][e] * h[j][e];
  return z;
}

// the states of sequences without tokens: `out` takes `in` (zeros without one)
template <typename E, int W>
__device__ __forceinline__ void pass_state(const ConvSiluParams &p, int n, int c0, const void *in, void *out) {
  if (!out || (p.cu ? p.cu[n + 1] != p.cu[n] : p.T != 0)) return;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const size_t at = ((size_t)n * (W - 1) + k) * p.C + c0;
    float x[CS_CH];
    if (in) load_ch<E>(static_cast<const E *>(in) + at, x);
    else zero_ch(x);
    store_ch<E>(static_cast<E *>(out) + at, x);
  }
}

template <typename E, int W>
__global__ __launch_bounds__(CS_THREADS) void conv_silu_kernel(ConvSiluParams p) {
  const uint32_t units = p.C / CS_CH, idx = blockIdx.x * CS_THREADS + threadIdx.x;
  const uint32_t run = idx / units;
  const int c0 = (idx % units) * CS_CH;
  if (run >= (uint32_t)p.runs) {
    if (run < (uint32_t)(p.runs + p.N)) pass_state<E, W>(p, run - p.runs, c0, p.s0, p.sT);
    return;
  }
  int64_t t = (int64_t)run * p.run;
  const int64_t t1 = min(t + p.run, p.TT);
  clear_tail<E>(p, p.y, t, t1, c0);
  const E *x = static_cast<const E *>(p.x);
  E *y = static_cast<E *>(p.y), *sT = static_cast<E *>(p.sT);
  float w[W][CS_CH], bias[CS_CH], h[W > 1 ? W - 1 : 1][CS_CH];
  load_weights<W>(p.w, p.bias, c0, w, bias);
  while (t < t1) {
    Seq s;
    s.find(p, t);
    if (s.nx <= t) break;  // behind the last sequence
    const int64_t end = min(t1, s.nx);
    load_history<E, W>(p, s, t, c0, h);
    for (; t < end; t += CS_BATCH) {
      Raw<E> xb[CS_BATCH];
#pragma unroll
      for (int i = 0; i < CS_BATCH; ++i) xb[i].load(x + (t + i) * p.C + c0, t + i < end);
#pragma unroll
      for (int i = 0; i < CS_BATCH; ++i) {
        if (t + i >= end) break;
        float xv[CS_CH], o[CS_CH];
        xb[i].get(xv);
#pragma unroll
        for (int e = 0; e < CS_CH; ++e) {
          const float z = conv_at<W>(w, bias, h, xv, e);
          o[e] = z * sigmoidf(z);
        }
        store_ch<E>(y + (t + i) * p.C + c0, o);
        if constexpr (W > 1) shift<W - 1>(h, xv);
      }
    }
    t = end;
    if (sT && end == s.nx) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) store_ch<E>(sT + ((int64_t)s.n * (W - 1) + k) * p.C + c0, h[k]);
    }
  }
}

// UL units (of CS_CH channels) by CS_THREADS / UL runs per workgroup.  A
// thread walks each sequence's part [a, b) of its run: step u computes dz[u]
// (zero behind the sequence) and emits the input at place u - (W - 1), which
// all dz up to u complete; a part that starts its sequence also emits the
// places before it, ds0.
template <typename E, int W, int UL>
__global__ __launch_bounds__(CS_THREADS, UL == 64 ? 4 : 3) void conv_silu_bwd_kernel(ConvSiluParams p) {
  constexpr int RUNS = CS_THREADS / UL, PER = UL * CS_CH * (W + 1);
  __shared__ float part[RUNS][PER];
  const int units = p.C / CS_CH, ul = threadIdx.x % UL;
  // a wave's lanes share their run where UL is a wave: its place, and all
  // branches on it, are then scalar
  const int rl = UL == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / UL) : threadIdx.x / UL;
  const int unit = blockIdx.x * UL + ul, c0 = unit * CS_CH;
  const bool act = unit < units;
  float dw[W][CS_CH], db[CS_CH];
#pragma unroll
  for (int j = 0; j < W; ++j) zero_ch(dw[j]);
  zero_ch(db);
  if ((int)blockIdx.y >= p.rows) {  // sequences without tokens
    const int64_t step = (int64_t)(gridDim.y - p.rows) * RUNS;
    if (act)
      for (int64_t n = ((int)blockIdx.y - p.rows) * RUNS + rl; n < p.N; n += step) pass_state<E, W>(p, (int)n, c0, p.dsT, p.ds0);
    return;
  }
  if (act) {
    int64_t a = ((int64_t)blockIdx.y * RUNS + rl) * p.run;
    const int64_t t1 = min(a + p.run, p.TT);
    clear_tail<E>(p, p.dx, a, t1, c0);
    const E *x = static_cast<const E *>(p.x), *dy = static_cast<const E *>(p.dy), *dsT = static_cast<const E *>(p.dsT);
    E *dx = static_cast<E *>(p.dx), *ds0 = static_cast<E *>(p.ds0);
    float w[W][CS_CH], bias[CS_CH], h[W > 1 ? W - 1 : 1][CS_CH], dz[W][CS_CH];
    load_weights<W>(p.w, p.bias, c0, w, bias);
    while (a < t1) {
      Seq s;
      s.find(p, a);
      if (s.nx <= a) break;
      const int64_t b = min(t1, s.nx), first = a == s.st ? a - (W - 1) : a;  // places [first, b)
      load_history<E, W>(p, s, a, c0, h);
#pragma unroll
      for (int k = 0; k < W; ++k) zero_ch(dz[k]);
      const int64_t lim = min(b + (W - 1), s.nx);  // rows behind it are not used
      Raw<E> xn[CS_BWD_BATCH], yn[CS_BWD_BATCH];
      auto fetch = [&](int64_t u0) {
#pragma unroll
        for (int i = 0; i < CS_BWD_BATCH; ++i) {
          const int64_t at = min(u0 + i, lim - 1) * p.C;
          xn[i].load(x + at + c0, true);
          yn[i].load(dy + at + c0, true);
        }
      };
      fetch(a);
      for (int64_t u0 = a; u0 < b + (W - 1); u0 += CS_BWD_BATCH) {
        Raw<E> xb[CS_BWD_BATCH], yb[CS_BWD_BATCH];
#pragma unroll
        for (int i = 0; i < CS_BWD_BATCH; ++i) {
          xb[i] = xn[i];
          yb[i] = yn[i];
        }
        fetch(u0 + CS_BWD_BATCH);
#pragma unroll
        for (int i = 0; i < CS_BWD_BATCH; ++i) {
          const int64_t u = u0 + i;
          if (u >= b + (W - 1)) break;
          float xv[CS_CH], g[CS_CH];
          xb[i].get(xv);
          yb[i].get(g);
          if (u < s.nx) {
#pragma unroll
            for (int e = 0; e < CS_CH; ++e) {
              const float z = conv_at<W>(w, bias, h, xv, e), sg = sigmoidf(z);
              g[e] *= sg * (1.f + z * (1.f - sg));
            }
          } else {
            zero_ch(g);
          }
          if (u < b) {
#pragma unroll
            for (int e = 0; e < CS_CH; ++e) {
              db[e] += g[e];
              dw[W - 1][e] += g[e] * xv[e];
#pragma unroll
              for (int j = 0; j < W - 1; ++j) dw[j][e] += g[e] * h[j][e];
            }
          }
          shift<W>(dz, g);
          if constexpr (W > 1) shift<W - 1>(h, xv);
          const int64_t q = u - (W - 1);
          if (q < first) continue;
          float o[CS_CH];
          // dz[k] is at u - (W - 1) + k = q + k
#pragma unroll
          for (int e = 0; e < CS_CH; ++e) {
            o[e] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) o[e] += w[j][e] * dz[W - 1 - j][e];
          }
          if (dsT && q >= s.nx - (W - 1)) {
            float d[CS_CH];
            load_ch<E>(dsT + ((int64_t)s.n * (W - 1) + (q - s.nx) + (W - 1)) * p.C + c0, d);
#pragma unroll
            for (int e = 0; e < CS_CH; ++e) o[e] += d[e];
          }
          if (q >= s.st) store_ch<E>(dx + q * p.C + c0, o);
          else if (ds0) store_ch<E>(ds0 + ((int64_t)s.n * (W - 1) + (q - s.st) + (W - 1)) * p.C + c0, o);
        }
      }
      a = b;
    }
  }
#pragma unroll
  for (int e = 0; e < CS_CH; ++e) {
    const int at = (ul * CS_CH + e) * (W + 1);
#pragma unroll
    for (int j = 0; j < W; ++j) part[rl][at + j] = dw[j][e];
    part[rl][at + W] = db[e];
  }
  __syncthreads();
  const int base = blockIdx.x * PER, n = p.C * (W + 1);
  for (int i = threadIdx.x; i < PER; i += CS_THREADS) {
    if (i >= n - base) break;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) sum += part[r][i];
    p.part[(size_t)blockIdx.y * n + base + i] = sum;
  }
}

// dw and dbias from the rows of partial sums
__global__ __launch_bounds__(CS_THREADS) void conv_silu_sum_kernel(ConvSiluParams p) {
  const int64_t n = (int64_t)p.C * (p.W + 1), col0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * SUM_COLS, i = col0 + threadIdx.x;
  const float a = column_sum(p.part, p.rows, n, col0);
  if (threadIdx.x >= SUM_COLS || i >= n) return;
  const int64_t c = i / (p.W + 1);
  const int j = (int)(i - c * (p.W + 1));
  if (j < p.W) p.dw[c * p.W + j] = a;
  else if (p.dbias) p.dbias[c] = a;
}

// one token of every sequence; the state takes the token's input
template <typename E, int W>
__global__ __launch_bounds__(CS_THREADS) void conv_silu_step_kernel(const E *x, const float *wt, const float *bs, E *state,
                                                                    E *y, uint32_t total, int C) {
  const uint32_t units = C / CS_CH, idx = blockIdx.x * CS_THREADS + threadIdx.x;
  if (idx >= total) return;
  const uint32_t n = idx / units;
  const int c0 = (idx % units) * CS_CH;
  float h[W > 1 ? W - 1 : 1][CS_CH], xv[CS_CH], w[W][CS_CH], bias[CS_CH], o[CS_CH];
  E *st = state + ((size_t)n * (W - 1)) * C + c0;
  load_ch<E>(x + (size_t)n * C + c0, xv);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) load_ch<E>(st + (size_t)k * C, h[k]);
  load_weights<W>(wt, bs, c0, w, bias);
#pragma unroll
  for (int e = 0; e < CS_CH; ++e) {
    const float z = conv_at<W>(w, bias, h, xv, e);
    o[e] = z * sigmoidf(z);
  }
  store_ch<E>(y + (size_t)n * C + c0, o);
  if constexpr (W > 1) {
#pragma unroll
    for (int k = 0; k + 1 < W - 1; ++k) store_ch<E>(st + (size_t)k * C, h[k + 1]);
    store_ch<E>(st + (size_t)(W - 2) * C, xv);
  }
}

// ------------------------------------------------------------------- host

bool aligned16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

dn_status check(int32_t B, int32_t T, int32_t H, int32_t D, int32_t W, int32_t n_seqs, int32_t dtype, const float *w,
                const int32_t *cu) {
  if (B <= 0 || T < 0 || H <= 0 || D <= 0 || n_seqs <= 0 || !w) return DN_EINVAL;
  if (dtype != DN_F32 && dtype != DN_BF16) return DN_EINVAL;
  if (cu ? B != 1 : n_seqs != B) return DN_EINVAL;
  if (D % 8 != 0 || W < 1 || W > 4) return DN_EUNSUPPORTED;
  if ((int64_t)H * D * (W + 1) > INT32_MAX) return DN_EUNSUPPORTED;
  return DN_OK;
}

// Units of a workgroup in the backward pass: 64 where a row has as many, else
// 16, so that short rows do not leave most lanes idle.
int unit_lanes(int C) { return C / CS_CH >= 64 ? 64 : 16; }

// Tokens of a run and rows of partial sums in the backward pass: 64 tokens where
// that gives each SIMD its four waves (4 x 4096 tokens of 4096 channels: 90 us,
// with 32 tokens 95 us), else 32, and longer ones beyond CS_MAX_ROWS rows.
void bwd_plan(int64_t TT, int C, int &run, int &rows) {
  const int64_t per = CS_THREADS / unit_lanes(C), least = TT / 64 * (C / CS_CH) >= 4 * 1024 * 64 ? 64 : 32;
  int64_t r = (TT + CS_MAX_ROWS * per - 1) / (CS_MAX_ROWS * per);
  r = r < least ? least : (r + 3) / 4 * 4;
  run = (int)r;
  rows = (int)((TT + r * per - 1) / (r * per));
}

template <typename E, int W>
void launch_fwd_w(const ConvSiluParams &p, unsigned grid, hipStream_t st) {
  hipLaunchKernelGGL((conv_silu_kernel<E, W>), dim3(grid), dim3(CS_THREADS), 0, st, p);
}
template <typename E>
void launch_fwd_e(const ConvSiluParams &p, unsigned grid, hipStream_t st) {
  switch (p.W) {
    case 1: return launch_fwd_w<E, 1>(p, grid, st);
    case 2: return launch_fwd_w<E, 2>(p, grid, st);
    case 3: return launch_fwd_w<E, 3>(p, grid, st);
    default: return launch_fwd_w<E, 4>(p, grid, st);
  }
}
template <typename E, int W>
void launch_bwd_w(const ConvSiluParams &p, hipStream_t st) {
  const int ul = unit_lanes(p.C), units = p.C / CS_CH, per = CS_THREADS / ul;
  // behind the rows, one workgroup row for every `per` sequences that may be empty,
  // or as many as a grid has (65535 with the rows), which then go on to further ones
  const int64_t groups = p.ds0 ? ((int64_t)p.N + per - 1) / per : 0, most = 65535 - p.rows;
  const dim3 grid((units + ul - 1) / ul, p.rows + (int)(groups < most ? groups : most));
  if (grid.y == 0) return;
  if (ul == 64) hipLaunchKernelGGL((conv_silu_bwd_kernel<E, W, 64>), grid, dim3(CS_THREADS), 0, st, p);
  else hipLaunchKernelGGL((conv_silu_bwd_kernel<E, W, 16>), grid, dim3(CS_THREADS), 0, st, p);
}
template <typename E>
void launch_bwd_e(const ConvSiluParams &p, hipStream_t st) {
  switch (p.W) {
    case 1: return launch_bwd_w<E, 1>(p, st);
    case 2: return launch_bwd_w<E, 2>(p, st);
    case 3: return launch_bwd_w<E, 3>(p, st);
    default: return launch_bwd_w<E, 4>(p, st);
  }
}
template <typename E, int W>
void launch_step_w(const void *x, const float *w, const float *b, void *state, void *y, uint32_t total, int C,
                   hipStream_t st) {
  hipLaunchKernelGGL((conv_silu_step_kernel<E, W>), dim3((total + CS_THREADS - 1) / CS_THREADS), dim3(CS_THREADS), 0, st,
                     static_cast<const E *>(x), w, b, static_cast<E *>(state), static_cast<E *>(y), total, C);
}
template <typename E>
void launch_step_e(int W, const void *x, const float *w, const float *b, void *state, void *y, uint32_t total, int C,
                   hipStream_t st) {
  switch (W) {
    case 1: return launch_step_w<E, 1>(x, w, b, state, y, total, C, st);
    case 2: return launch_step_w<E, 2>(x, w, b, state, y, total, C, st);
    case 3: return launch_step_w<E, 3>(x, w, b, state, y, total, C, st);
    default: return launch_step_w<E, 4>(x, w, b, state, y, total, C, st);
  }
}

}  // namespace
}  // namespace dn

using namespace dn;

extern "C" dn_status dn_conv_silu(int32_t B, int32_t T, int32_t H, int32_t D, int32_t W, int32_t n_seqs, int32_t dtype,
                                  const void *x, const float *w, const float *bias, const void *s0,
                                  const int32_t *cu_seqlens, void *y, void *sT, hipStream_t stream) {
  const bool zero_tail = cu_seqlens && (dtype & DN_ZERO_TAIL);
  dtype &= ~DN_ZERO_TAIL;
  const dn_status st = check(B, T, H, D, W, n_seqs, dtype, w, cu_seqlens);
  if (st != DN_OK) return st;
  if (!aligned16(s0) || !aligned16(sT) || !aligned16(w) || !aligned16(bias)) return DN_EINVAL;
  if (T > 0 && (!x || !y || !aligned16(x) || !aligned16(y))) return DN_EINVAL;
  ConvSiluParams p = {};
  p.x = x;
  p.s0 = s0;
  p.w = w;
  p.bias = bias;
  p.cu = cu_seqlens;
  p.y = y;
  p.sT = W > 1 ? sT : nullptr;
  p.TT = (int64_t)B * T;
  p.T = T;
  p.N = n_seqs;
  p.C = H * D;
  p.W = W;
  p.zero_tail = zero_tail;
  // runs of 32 tokens, or of 8 where those would leave the CUs without 8 waves each
  const int64_t units = p.C / CS_CH;
  p.run = (p.TT + 31) / 32 * units >= 256 * 8 * 64 ? 32 : 8;
  const int64_t runs = (p.TT + p.run - 1) / p.run, total = (runs + (p.sT ? n_seqs : 0)) * units;
  if (total > INT32_MAX) return DN_EUNSUPPORTED;
  if (total == 0) return DN_OK;
  p.runs = (int)runs;
  const unsigned grid = (unsigned)((total + CS_THREADS - 1) / CS_THREADS);
  if (dtype == DN_BF16) launch_fwd_e<bf16>(p, grid, stream);
  else launch_fwd_e<float>(p, grid, stream);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" size_t dn_conv_silu_bwd_workspace(int32_t B, int32_t T, int32_t H, int32_t D, int32_t W) {
  if (B <= 0 || T <= 0 || H <= 0 || D <= 0 || W < 1 || W > 4 || (int64_t)H * D * (W + 1) > INT32_MAX) return 0;
  int run, rows;
  bwd_plan((int64_t)B * T, H * D, run, rows);
  return 4 * (size_t)rows * H * D * (W + 1);
}

extern "C" dn_status dn_conv_silu_bwd(int32_t B, int32_t T, int32_t H, int32_t D, int32_t W, int32_t n_seqs,
                                      int32_t dtype, const void *x, const float *w, const float *bias, const void *s0,
                                      const int32_t *cu_seqlens, const void *dy, const void *dsT, void *dx, float *dw,
                                      float *dbias, void *ds0, void *workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
  const bool zero_tail = cu_seqlens && (dtype & DN_ZERO_TAIL);
  dtype &= ~DN_ZERO_TAIL;
  const dn_status st = check(B, T, H, D, W, n_seqs, dtype, w, cu_seqlens);
  if (st != DN_OK) return st;
  if (!dw || !aligned16(s0) || !aligned16(dsT) || !aligned16(ds0) || !aligned16(w) || !aligned16(bias)) return DN_EINVAL;
  if (T > 0 && (!x || !dy || !dx || !aligned16(x) || !aligned16(dy) || !aligned16(dx))) return DN_EINVAL;
  ConvSiluParams p = {};
  p.x = x;
  p.s0 = s0;
  p.dy = dy;
  p.dsT = dsT;
  p.w = w;
  p.bias = bias;
  p.cu = cu_seqlens;
  p.dx = dx;
  p.ds0 = W > 1 ? ds0 : nullptr;
  p.dw = dw;
  p.dbias = dbias;
  p.part = static_cast<float *>(workspace);
  p.TT = (int64_t)B * T;
  p.T = T;
  p.N = n_seqs;
  p.C = H * D;
  p.W = W;
  p.zero_tail = zero_tail;
  bwd_plan(p.TT, p.C, p.run, p.rows);
  if (p.rows > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < dn_conv_silu_bwd_workspace(B, T, H, D, W)))
    return DN_ENOWS;
  if (dtype == DN_BF16) launch_bwd_e<bf16>(p, stream);
  else launch_bwd_e<float>(p, stream);
  if (hipGetLastError() != hipSuccess) return DN_EHIP;
  // A grid has fewer than 2^32 threads in one direction (one of 2^32 + 32768 ran
  // 32768, without an error): lines of 2^20 workgroups.
  const int64_t sums = ((int64_t)p.C * (W + 1) + SUM_COLS - 1) / SUM_COLS, line = sums < 1 << 20 ? sums : 1 << 20;
  hipLaunchKernelGGL(conv_silu_sum_kernel, dim3((unsigned)line, (unsigned)((sums + line - 1) / line)), dim3(CS_THREADS), 0,
                     stream, p);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" dn_status dn_conv_silu_step(int32_t B, int32_t H, int32_t D, int32_t W, int32_t dtype, const void *x,
                                       const float *w, const float *bias, void *state, void *y, hipStream_t stream) {
  const dn_status st = check(B, 1, H, D, W, B, dtype, w, nullptr);
  if (st != DN_OK) return st;
  if (!x || !y || (W > 1 && !state) || !aligned16(x) || !aligned16(y) || !aligned16(state) || !aligned16(w) ||
      !aligned16(bias))
    return DN_EINVAL;
  const int64_t total = (int64_t)B * (H * D / CS_CH);
  if (total > INT32_MAX) return DN_EUNSUPPORTED;
  if (dtype == DN_BF16) launch_step_e<bf16>(W, x, w, bias, state, y, (uint32_t)total, H * D, stream);
  else launch_step_e<float>(W, x, w, bias, state, y, (uint32_t)total, H * D, stream);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}
