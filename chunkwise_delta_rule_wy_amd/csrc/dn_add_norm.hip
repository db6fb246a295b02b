// The residual's addition in front of a layer, with dropout and root-mean-square
// norm, its backward pass, and the form that leaves the rows in 8 bits, for
// gfx950.  Per row of D values:
//
//   h = residual + d x,        d = 0 or 1 / (1 - p), a value's own
//   y = n w,                   n = h r,  r = (mean h^2 + eps)^-1/2
//
//   dresidual = dh + r (dn - n mean(dn n)),   dn = dy w
//   dx = d dresidual,          dw = sum dy n
//
// h is rounded once, as it is stored, and the norm is that of the stored values:
// the backward pass reads nothing else of the forward pass.  A row sits in
// registers of a group of lanes (Row), so that every tensor crosses HBM once.
//
// The mask is never stored: both passes compute it from the seed and a value's
// place with Philox4x32 (Salmon et al., "Parallel random numbers: as easy as 1,
// 2, 3", 2011), in its form of 7 rounds, the fewest that pass the paper's tests.
// A block of 128 bits serves the 8 values of a unit, 16 bits each.
#include "dn.h"
#include "dn_rows.h"

namespace dn {
namespace {

constexpr int AN_THREADS = ROW_THREADS;
constexpr int AN_MAX_D = 8192;
// Workgroups: all that the CUs hold forwards, two per CU backwards, which load a row
// ahead and leave as many rows of partial sums (16384 rows of 4096 bf16 values with
// dropout, before the stores went past the caches: 136 us, with four per CU 143; without
// the row ahead 201 us), each going on to further rows.  Both are bound by memory: these
// rows take 102 us forwards, 125 backwards and 97 in 8 bits at best (medians 103, 131 and
// 99), that is 5.3, 5.4 and 4.8 TB/s, where a copy reaches 5.1.
constexpr int AN_FWD_BLOCKS = 2048, AN_BWD_BLOCKS = 512;

struct AddNormParams {
  const void *x, *res, *dy, *dh;  // res, dh may be null
  const float *w;                 // null (norm8): no norm
  const uint64_t *seed;           // key and stream
  void *y, *h, *dx, *dres;        // h, dx, dres may be null
  float *scale, *part, *dw;
  int64_t rows;  // below 2^31
  int D, blocks;
  uint32_t drop;  // a value is dropped where its 16 bits are below
  float eps, keep;
};

struct Bits128 {
  uint32_t w[4];
};

__device__ __forceinline__ Bits128 philox7(uint64_t key, uint64_t stream, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)stream, c3 = (uint32_t)(stream >> 32);
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {c0, c1, c2, c3};
}

// x[i] *= d, for the values of `row` that a lane holds
template <typename RW, int LPR, int K>
__device__ __forceinline__ void drop_out(const AddNormParams &p, uint64_t key, uint64_t stream, int64_t row, int lane,
                                         float (&x)[RW::N]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = RW::col(k, lane);
    const Bits128 b = philox7(key, stream, (uint64_t)row * (uint32_t)(p.D >> 3) + (uint32_t)(c >> 3));
#pragma unroll
    for (int e = 0; e < RW::V; ++e) {
      // a unit of four fp32 values takes its half of the block
      const uint32_t w = RW::V == 8 ? b.w[e >> 1] : c & 4 ? b.w[2 + (e >> 1)] : b.w[e >> 1];
      x[k * RW::V + e] *= (e & 1 ? w >> 16 : w & 0xffffu) >= p.drop ? p.keep : 0.f;
    }
  }
}

// h = residual + d x, rounded to R, stored where asked for
template <typename E, typename R, int LPR, int K, bool DROP>
__device__ __forceinline__ void add_row(const AddNormParams &p, uint64_t key, uint64_t stream, int64_t row, int lane,
                                        float (&h)[Row<E, LPR, K>::N]) {
  using RW = Row<E, LPR, K>;
  const int64_t at = row * p.D;
  RW::load(static_cast<const E *>(p.x) + at, lane, p.D, h);
  if (p.res) {
    float res[RW::N];
    RW::load(static_cast<const R *>(p.res) + at, lane, p.D, res);
    if (DROP) drop_out<RW, LPR, K>(p, key, stream, row, lane, h);
#pragma unroll
    for (int i = 0; i < RW::N; ++i) h[i] += res[i];
  } else if (DROP) {
    drop_out<RW, LPR, K>(p, key, stream, row, lane, h);
  }
#pragma unroll
  for (int i = 0; i < RW::N; ++i) h[i] = to_f<R>(to_e<R>(h[i]));
  if (p.h) RW::template store<true>(static_cast<R *>(p.h) + at, lane, p.D, h);
}

template <int LPR, int N>
__device__ __forceinline__ float row_rsqrt(const AddNormParams &p, const float (&h)[N], float (*buf)[AN_THREADS / 64],
                                           int &turn) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) ss += h[i] * h[i];
  return rsqrtf(lanes_sum<LPR>(ss, buf, turn) / (float)p.D + p.eps);
}

template <typename E, typename R, int LPR, int K, bool DROP>
__global__ __launch_bounds__(AN_THREADS) void add_norm_kernel(AddNormParams p) {
  using RW = Row<E, LPR, K>;
  __shared__ float buf[2][AN_THREADS / 64];
  int turn = 0;
  const int lane = threadIdx.x % LPR;
  const uint64_t key = DROP ? p.seed[0] : 0, stream = DROP ? p.seed[1] : 0;
  float w[RW::N];
  RW::load_w(p.w, lane, p.D, w);
  for (int64_t row = (int64_t)blockIdx.x * (AN_THREADS / LPR) + threadIdx.x / LPR; row < p.rows;
       row += (int64_t)gridDim.x * (AN_THREADS / LPR)) {
    float h[RW::N];
    add_row<E, R, LPR, K, DROP>(p, key, stream, row, lane, h);
    const float r = row_rsqrt<LPR>(p, h, buf, turn);
#pragma unroll
    for (int i = 0; i < RW::N; ++i) h[i] = h[i] * r * w[i];
    RW::template store<true>(static_cast<E *>(p.y) + row * p.D, lane, p.D, h);
  }
}

// The rows in 8 bits (4 exponent and 3 mantissa bits, largest value 448) with a
// scale each: q = y / scale rounded to fp32 and then to 8 bits, scale = max |y| / 448.
// Rows of zeros have the scale 1e-30 / 448, whose inverse is still finite.
//
// The quotients are those of an fp32 division: a product with the rounded inverse takes
// some bf16 values of a row that is not normed (0.05 % in rows of 64, 0.03 % in rows of 4096),
// whose quotients lie on a half, to the other side of it.  1 / s = inv + low to some 46
// bits, so that q is one of the two fp32 numbers around the quotient; its remainder v - q s
// then is exact, and q + remainder inv, rounded, is the quotient rounded (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// In us, with the inverse alone and with the compiler's division: 16384 normed rows of 4096
// bf16 values 99 (98, 99), 65536 of 1024 100 (99, 102), 8192 rows of 8192 without norm or residual
// 34.7 (32.9, 41.5).
constexpr float TOP8 = 448.f, LEAST8 = 1e-30f;

template <typename E, typename R, int LPR, int K, bool NORM>
__global__ __launch_bounds__(AN_THREADS) void norm8_kernel(AddNormParams p) {
  using RW = Row<E, LPR, K>;
  __shared__ float buf[2][AN_THREADS / 64];
  int turn = 0;
  const int lane = threadIdx.x % LPR;
  float w[RW::N];
  if (NORM) RW::load_w(p.w, lane, p.D, w);
  for (int64_t row = (int64_t)blockIdx.x * (AN_THREADS / LPR) + threadIdx.x / LPR; row < p.rows;
       row += (int64_t)gridDim.x * (AN_THREADS / LPR)) {
    float h[RW::N];
    add_row<E, R, LPR, K, false>(p, 0, 0, row, lane, h);
    float top = LEAST8;
    if (NORM) {
      const float r = row_rsqrt<LPR>(p, h, buf, turn);
      // an infinity becomes NaN, which a maximum passes over, and all else 0: it is
      // looked for itself
      if (!(r > 0.f)) {
#pragma unroll
        for (int i = 0; i < RW::N; ++i) top = fabsf(h[i]) == __builtin_inff() ? __builtin_inff() : top;
      }
#pragma unroll
      for (int i = 0; i < RW::N; ++i) h[i] = h[i] * r * w[i];
    }
#pragma unroll
    for (int i = 0; i < RW::N; ++i) top = fmaxf(top, fabsf(h[i]));
    const float scale = lanes_sum<LPR, true>(top, buf, turn) / TOP8;
    float s = scale;
    if (s < 0x1p-90f) {  // the remainders of such rows would fall below fp32
      s *= 0x1p64f;
#pragma unroll
      for (int i = 0; i < RW::N; ++i) h[i] *= 0x1p64f;
    }
    float inv = 1.f / s, low = __builtin_fmaf(-inv, s, 1.f) * inv;
    if (s == __builtin_inff()) {  // v / s is 0, and NaN for an infinite v; a normed row is NaN as a whole
      inv = low = NORM ? __builtin_nanf("") : 0.f;
      s = 1.f;
    }
    const auto quotient = [&](float v) {
      const float q = __builtin_fmaf(v, inv, v * low);
      return __builtin_fmaf(__builtin_fmaf(-q, s, v), inv, q);
    };
    uint8_t *out = static_cast<uint8_t *>(p.y) + row * p.D;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = RW::col(k, lane);
      if (c >= p.D) continue;
      uint32_t q[RW::V / 4];
#pragma unroll
      for (int j = 0; j < RW::V / 4; ++j) {
        const float *v = h + k * RW::V + 4 * j;
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[0]), quotient(v[1]), 0, false);
        q[j] = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[2]), quotient(v[3]), lo, true);
      }
      if constexpr (RW::V == 8) __builtin_nontemporal_store((u32x2){q[0], q[1]}, reinterpret_cast<u32x2 *>(out + c));
      else __builtin_nontemporal_store(q[0], reinterpret_cast<uint32_t *>(out + c));
    }
    if (lane == 0) p.scale[row] = scale;
  }
}

template <typename E, typename R, int LPR, int K, bool DROP>
__global__ __launch_bounds__(AN_THREADS) void add_norm_bwd_kernel(AddNormParams p) {
  using RW = Row<E, LPR, K>;
  constexpr int GROUPS = AN_THREADS / LPR, PER = LPR * RW::N;
  __shared__ f32x2 buf[2][AN_THREADS / 64];
  __shared__ float part[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? PER : 1];
  int turn = 0;
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const uint64_t key = DROP ? p.seed[0] : 0, stream = DROP ? p.seed[1] : 0;
  float w[RW::N], dw[RW::N];
  RW::load_w(p.w, lane, p.D, w);
#pragma unroll
  for (int i = 0; i < RW::N; ++i) dw[i] = 0.f;
  const float inv = 1.f / (float)p.D;
  // the next row is loaded while this one is worked on; without dh a row of h stands
  // in for it, and for the rows behind the last one that one, so that nothing branches
  // around the loads
  RawRow<E, R, LPR, K> rh, rg;
  RawRow<E, E, LPR, K> ry;
  const R *h_in = static_cast<const R *>(p.h), *g_in = static_cast<const R *>(p.dh ? p.dh : p.h);
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t row = (int64_t)blockIdx.x * GROUPS + grp;
  const auto load = [&](int64_t r) {
    const int64_t at = min(r, p.rows - 1) * p.D;
    rh.load(h_in + at, lane, p.D);
    ry.load(static_cast<const E *>(p.dy) + at, lane, p.D);
    rg.load(g_in + at, lane, p.D);
  };
  if (p.rows > 0) load(row);
  for (; row < p.rows; row += step) {
    const int64_t at = row * p.D;
    float h[RW::N], dy[RW::N], g[RW::N];
    rh.get(lane, p.D, h);
    ry.get(lane, p.D, dy);
    rg.get(lane, p.D, g);
    load(row + step);
    f32x2 sums = {0.f, 0.f};  // h^2, and dn n / r
#pragma unroll
    for (int i = 0; i < RW::N; ++i) sums = (f32x2){sums[0] + h[i] * h[i], sums[1] + dy[i] * w[i] * h[i]};
    sums = lanes_sum2<LPR>(sums, buf, turn);
    const float r = rsqrtf(sums[0] * inv + p.eps);
    const float mean = sums[1] * r * inv;
#pragma unroll
    for (int i = 0; i < RW::N; ++i) {
      const float n = h[i] * r;
      g[i] = (p.dh ? g[i] : 0.f) + r * (dy[i] * w[i] - n * mean);
      dw[i] += dy[i] * n;
    }
    if (p.dres) RW::template store<true>(static_cast<R *>(p.dres) + at, lane, p.D, g);
    if (p.dx) {
      if (DROP) drop_out<RW, LPR, K>(p, key, stream, row, lane, g);
      RW::template store<true>(static_cast<E *>(p.dx) + at, lane, p.D, g);
    }
  }
  float *out = p.part + (size_t)blockIdx.x * p.D;
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < RW::V; ++e) {
        const int c = RW::col(k, lane) + e;
        if (c < p.D) out[c] = dw[k * RW::V + e];
      }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < RW::V; ++e) part[grp][RW::col(k, lane) + e] = dw[k * RW::V + e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += AN_THREADS) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) s += part[i][c];
      out[c] = s;
    }
  }
}

// dw from the workgroups' partial sums, in a fixed order
__global__ __launch_bounds__(AN_THREADS) void add_norm_sum_kernel(AddNormParams p) {
  const int col0 = blockIdx.x * SUM_COLS, c = col0 + threadIdx.x;
  const float a = column_sum(p.part, p.blocks, p.D, col0);
  if (threadIdx.x < SUM_COLS && c < p.D) p.dw[c] = a;
}

// ------------------------------------------------------------------- host

bool aligned16(std::initializer_list<const void *> ps) {
  for (const void *q : ps)
    if (reinterpret_cast<uintptr_t>(q) & 15u) return false;
  return true;
}

dn_status check(int64_t rows, int32_t D, int32_t dtype, int32_t res_dtype) {
  if (rows < 0 || D <= 0) return DN_EINVAL;
  if ((dtype != DN_F32 && dtype != DN_BF16) || (res_dtype != DN_F32 && res_dtype != dtype)) return DN_EINVAL;
  if (D % 8 != 0 || D > AN_MAX_D || rows > INT32_MAX) return DN_EUNSUPPORTED;
  return DN_OK;
}

// p as 16 bits: a value is dropped with probability drop / 65536
dn_status set_drop(AddNormParams &a, double p, const uint64_t *seed) {
  if (!(p >= 0.0 && p < 1.0)) return DN_EINVAL;
  a.drop = (uint32_t)__builtin_nearbyint(p * 65536.0);
  if (a.drop > 65535u) return DN_EUNSUPPORTED;
  if (a.drop && !seed) return DN_EINVAL;
  a.keep = (float)(65536.0 / (65536.0 - a.drop));
  a.seed = seed;
  return DN_OK;
}

int fwd_blocks(int64_t rows, int per) {
  const int64_t groups = (rows + per - 1) / per;
  return (int)(groups < AN_FWD_BLOCKS ? groups : AN_FWD_BLOCKS);
}

int bwd_blocks(int64_t rows) { return rows < 1 ? 1 : (int)(rows < AN_BWD_BLOCKS ? rows : AN_BWD_BLOCKS); }

enum Pass { FORWARD, BACKWARD, EIGHT };

template <typename E, typename R, int LPR, int K>
void launch_lk(const AddNormParams &p, Pass pass, hipStream_t st) {
  const dim3 fwd(fwd_blocks(p.rows, AN_THREADS / LPR)), bwd(p.blocks), thr(AN_THREADS);
  const bool drop = p.drop > 0;
  if (pass == FORWARD) {
    if (drop) hipLaunchKernelGGL((add_norm_kernel<E, R, LPR, K, true>), fwd, thr, 0, st, p);
    else hipLaunchKernelGGL((add_norm_kernel<E, R, LPR, K, false>), fwd, thr, 0, st, p);
  } else if (pass == BACKWARD) {
    if (drop) hipLaunchKernelGGL((add_norm_bwd_kernel<E, R, LPR, K, true>), bwd, thr, 0, st, p);
    else hipLaunchKernelGGL((add_norm_bwd_kernel<E, R, LPR, K, false>), bwd, thr, 0, st, p);
  } else {
    if (p.w) hipLaunchKernelGGL((norm8_kernel<E, R, LPR, K, true>), fwd, thr, 0, st, p);
    else hipLaunchKernelGGL((norm8_kernel<E, R, LPR, K, false>), fwd, thr, 0, st, p);
  }
}

// Lanes per row and 16-byte units per lane, by the row's units, as the gated norm
// chooses them: the fewest lanes that hold a row with one unit each, from 65 to
// 128 units a wave with two, then the workgroup.
template <typename E, typename R>
void launch_er(const AddNormParams &p, Pass pass, hipStream_t st) {
  const int u = p.D / Vec16<E>::N;
  if (u <= 8) launch_lk<E, R, 8, 1>(p, pass, st);
  else if (u <= 16) launch_lk<E, R, 16, 1>(p, pass, st);
  else if (u <= 32) launch_lk<E, R, 32, 1>(p, pass, st);
  else if (u <= 64) launch_lk<E, R, 64, 1>(p, pass, st);
  else if (u <= 128) launch_lk<E, R, 64, 2>(p, pass, st);
  else if (u <= 256) launch_lk<E, R, 256, 1>(p, pass, st);
  else if (u <= 512) launch_lk<E, R, 256, 2>(p, pass, st);
  else if (u <= 1024) launch_lk<E, R, 256, 4>(p, pass, st);
  else if constexpr (sizeof(E) == 4) launch_lk<E, R, 256, 8>(p, pass, st);  // bf16 ends at 8192 / 8 units
}

dn_status launch(const AddNormParams &p, int dtype, int res_dtype, Pass pass, hipStream_t st) {
  if (dtype == DN_F32) launch_er<float, float>(p, pass, st);
  else if (res_dtype == DN_F32) launch_er<bf16, float>(p, pass, st);
  else launch_er<bf16, bf16>(p, pass, st);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}

}  // namespace
}  // namespace dn

using namespace dn;

extern "C" dn_status dn_add_norm(int64_t rows, int32_t D, int32_t dtype, int32_t res_dtype, const void *x,
                                 const void *residual, const float *w, float eps, double p, const uint64_t *seed, void *y,
                                 void *h, hipStream_t stream) {
  dn_status st = check(rows, D, dtype, res_dtype);
  if (st != DN_OK) return st;
  AddNormParams a = {};
  st = set_drop(a, p, seed);
  if (st != DN_OK) return st;
  if (!w) return DN_EINVAL;
  if (rows == 0) return DN_OK;
  if (!x || !y || !aligned16({x, residual, y, h})) return DN_EINVAL;
  a.x = x;
  a.res = residual;
  a.w = w;
  a.y = y;
  a.h = h;
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  return launch(a, dtype, res_dtype, FORWARD, stream);
}

extern "C" size_t dn_add_norm_bwd_workspace(int64_t rows, int32_t D) {
  if (rows < 0 || D <= 0 || D > AN_MAX_D) return 0;
  return 4 * (size_t)bwd_blocks(rows) * D;
}

extern "C" dn_status dn_add_norm_bwd(int64_t rows, int32_t D, int32_t dtype, int32_t res_dtype, const void *h,
                                     const float *w, float eps, double p, const uint64_t *seed, const void *dy,
                                     const void *dh, void *dx, void *dres, float *dw, void *workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  dn_status st = check(rows, D, dtype, res_dtype);
  if (st != DN_OK) return st;
  AddNormParams a = {};
  st = set_drop(a, p, seed);
  if (st != DN_OK) return st;
  if (!w || !dw) return DN_EINVAL;
  if (rows > 0 && (!h || !dy || !aligned16({h, dy, dh, dx, dres}))) return DN_EINVAL;
  if (!workspace || !aligned16({workspace}) || workspace_bytes < dn_add_norm_bwd_workspace(rows, D)) return DN_ENOWS;
  a.h = const_cast<void *>(h);
  a.w = w;
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.dres = dres;
  a.dw = dw;
  a.part = static_cast<float *>(workspace);
  a.rows = rows;
  a.D = D;
  a.blocks = bwd_blocks(rows);
  a.eps = eps;
  st = launch(a, dtype, res_dtype, BACKWARD, stream);
  if (st != DN_OK) return st;
  hipLaunchKernelGGL(add_norm_sum_kernel, dim3((D + SUM_COLS - 1) / SUM_COLS), dim3(AN_THREADS), 0, stream, a);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" dn_status dn_norm8(int64_t rows, int32_t D, int32_t dtype, int32_t res_dtype, const void *x,
                              const void *residual, const float *w, float eps, void *y, float *scale, void *h,
                              hipStream_t stream) {
  const dn_status st = check(rows, D, dtype, res_dtype);
  if (st != DN_OK) return st;
  if (rows == 0) return DN_OK;
  if (!x || !y || !scale || !aligned16({x, residual, y, h})) return DN_EINVAL;
  AddNormParams a = {};
  a.x = x;
  a.res = residual;
  a.w = w;
  a.y = y;
  a.scale = scale;
  a.h = h;
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  return launch(a, dtype, res_dtype, EIGHT, stream);
}
