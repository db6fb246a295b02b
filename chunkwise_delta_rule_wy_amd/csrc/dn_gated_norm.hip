// Gated root-mean-square norm of the rows behind a token mixer and its
// backward, for gfx950.  Per row of D values, with g = z sigmoid(z):
//
//   gate after the norm:   n = x r,    r = (mean x^2 + eps)^-1/2,      y = n w g
//   gate before the norm:  n = x g r,  r = (mean (x g)^2 + eps)^-1/2,  y = n w
//
//   du = r (dn - n mean(dn n)),   dn = dy w g (after) or dy w (before)
//   after:   dx = du,    dz = dy w n g'(z),   dw = sum dy n g
//   before:  dx = du g,  dz = du x g'(z),     dw = sum dy n
//
// with g'(z) = sigmoid(z) (1 + z (1 - sigmoid(z))).  A row sits in registers
// of a group of LPR lanes (one wave's part, or the whole workgroup for wide
// rows), K units of 16 bytes per lane, so that every tensor crosses HBM once,
// which bounds both passes: 262144 rows of 256 values in bf16 take 80 us
// forwards (403 MB, 5.0 TB/s) and 117 us backwards (671 MB, 5.7 TB/s), the rates
// of large copies.  Two, four or eight rows per lane group with all loads first
// are slower (91, 119, 167 us forwards: fewer waves).
// The weights' gradient is summed in registers over the rows that a workgroup
// takes (all of one weight row), in LDS over its lane groups and by a second
// kernel over the workgroups, in a fixed order.
#include "dn.h"
#include "dn_rows.h"

namespace dn {
namespace {

constexpr int GN_THREADS = ROW_THREADS;
// Workgroups: four per CU backwards (as many rows of partial sums), and up to
// eight forwards, all that a CU holds, which then go on to further rows
// (262144 rows of 256 values, bf16: 80 us, with four per CU 114 us, with
// workgroups for all rows 83 us).
constexpr int GN_BLOCKS = 1024, GN_FWD_BLOCKS = 2048;
constexpr int GN_MAX_D = 8192;

struct GatedNormParams {
  const void *x, *z, *dy;
  const float *w;
  void *y, *dx, *dz;
  float *part, *dw;
  int64_t rows;  // rows of x, below 2^31
  int D, R;      // R weight rows: row i uses weight row i % R
  int blocks;    // backward: workgroups per weight row
  float eps;
};

__device__ __forceinline__ float sigmoidf(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

template <typename E, int LPR, int K, bool FIRST>
__global__ __launch_bounds__(GN_THREADS) void gated_norm_kernel(GatedNormParams p) {
  using RW = Row<E, LPR, K>;
  __shared__ float buf[2][GN_THREADS / 64];
  int turn = 0;
  const int lane = threadIdx.x % LPR;
  // a row's lanes stay together, so that the sums over them are whole
  for (int64_t row = (int64_t)blockIdx.x * (GN_THREADS / LPR) + threadIdx.x / LPR; row < p.rows;
       row += (int64_t)gridDim.x * (GN_THREADS / LPR)) {
    float x[RW::N], z[RW::N], w[RW::N];
    RW::load(static_cast<const E *>(p.x) + row * p.D, lane, p.D, x);
    RW::load(static_cast<const E *>(p.z) + row * p.D, lane, p.D, z);
    RW::load_w(p.w + (size_t)((uint32_t)row % (uint32_t)p.R) * p.D, lane, p.D, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < RW::N; ++i) {
      z[i] *= sigmoidf(z[i]);
      if (FIRST) x[i] *= z[i];
      ss += x[i] * x[i];
    }
    const float r = rsqrtf(lanes_sum<LPR>(ss, buf, turn) / (float)p.D + p.eps);
#pragma unroll
    for (int i = 0; i < RW::N; ++i) x[i] = x[i] * r * w[i] * (FIRST ? 1.f : z[i]);
    RW::store(static_cast<E *>(p.y) + row * p.D, lane, p.D, x);
  }
}

template <typename E, int LPR, int K, bool FIRST>
__global__ __launch_bounds__(GN_THREADS) void gated_norm_bwd_kernel(GatedNormParams p) {
  using RW = Row<E, LPR, K>;
  constexpr int GROUPS = GN_THREADS / LPR, PER = LPR * RW::N;
  __shared__ float buf[2][GN_THREADS / 64];
  __shared__ float part[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? PER : 1];
  int turn = 0;
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int wr = blockIdx.x / p.blocks, blk = blockIdx.x % p.blocks;
  const int64_t per_w = p.rows / p.R;  // rows that share a weight row
  float w[RW::N], dw[RW::N];
  RW::load_w(p.w + (size_t)wr * p.D, lane, p.D, w);
#pragma unroll
  for (int i = 0; i < RW::N; ++i) dw[i] = 0.f;
  const float inv = 1.f / (float)p.D;
  for (int64_t i0 = (int64_t)blk * GROUPS + grp; i0 < per_w; i0 += (int64_t)p.blocks * GROUPS) {
    const int64_t at = (i0 * p.R + wr) * p.D;
    float x[RW::N], z[RW::N], dy[RW::N];
    RW::load(static_cast<const E *>(p.x) + at, lane, p.D, x);
    RW::load(static_cast<const E *>(p.z) + at, lane, p.D, z);
    RW::load(static_cast<const E *>(p.dy) + at, lane, p.D, dy);
    float ss = 0.f, dot = 0.f;
    float sg[RW::N];
#pragma unroll
    for (int i = 0; i < RW::N; ++i) {
      sg[i] = sigmoidf(z[i]);
      const float gate = z[i] * sg[i], u = FIRST ? x[i] * gate : x[i];
      ss += u * u;
      dot += dy[i] * w[i] * (FIRST ? u : gate * u);  // dn n / r
    }
    ss = lanes_sum<LPR>(ss, buf, turn);
    dot = lanes_sum<LPR>(dot, buf, turn);
    const float r = rsqrtf(ss * inv + p.eps);
    const float mean = dot * r * inv;
#pragma unroll
    for (int i = 0; i < RW::N; ++i) {
      const float gate = z[i] * sg[i], dgate = sg[i] * (1.f + z[i] * (1.f - sg[i]));
      const float u = FIRST ? x[i] * gate : x[i], n = u * r;
      const float dn = FIRST ? dy[i] * w[i] : dy[i] * w[i] * gate;
      const float du = r * (dn - n * mean);
      dw[i] += FIRST ? dy[i] * n : dy[i] * n * gate;
      z[i] = FIRST ? du * x[i] * dgate : dy[i] * w[i] * n * dgate;
      x[i] = FIRST ? du * gate : du;
    }
    RW::store(static_cast<E *>(p.dx) + at, lane, p.D, x);
    RW::store(static_cast<E *>(p.dz) + at, lane, p.D, z);
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
    for (int c = threadIdx.x; c < p.D; c += GN_THREADS) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) s += part[i][c];
      out[c] = s;
    }
  }
}

// dw from the workgroups' partial sums
__global__ __launch_bounds__(GN_THREADS) void gated_norm_sum_kernel(GatedNormParams p) {
  const int wr = blockIdx.x, col0 = blockIdx.y * SUM_COLS, c = col0 + threadIdx.x;
  const float a = column_sum(p.part + (size_t)wr * p.blocks * p.D, p.blocks, p.D, col0);
  if (threadIdx.x < SUM_COLS && c < p.D) p.dw[(size_t)wr * p.D + c] = a;
}

// ------------------------------------------------------------------- host

bool aligned16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

dn_status check(int64_t rows, int32_t D, int32_t R, int32_t dtype, const float *w) {
  if (rows < 0 || D <= 0 || R <= 0 || !w || rows % R != 0) return DN_EINVAL;
  if (dtype != DN_F32 && dtype != DN_BF16) return DN_EINVAL;
  if (D % 8 != 0 || D > GN_MAX_D) return DN_EUNSUPPORTED;
  return DN_OK;
}

int block_count(int64_t rows, int32_t R) {
  int64_t n = GN_BLOCKS / R;
  if (n > rows / R) n = rows / R;
  return n < 1 ? 1 : (int)n;
}

template <typename E, int LPR, int K>
void launch_lk(const GatedNormParams &p, bool first, bool bwd, hipStream_t st) {
  if (bwd) {
    const dim3 grid((unsigned)(p.R * p.blocks));
    if (first) hipLaunchKernelGGL((gated_norm_bwd_kernel<E, LPR, K, true>), grid, dim3(GN_THREADS), 0, st, p);
    else hipLaunchKernelGGL((gated_norm_bwd_kernel<E, LPR, K, false>), grid, dim3(GN_THREADS), 0, st, p);
  } else {
    constexpr int per = GN_THREADS / LPR;
    const int64_t groups = (p.rows + per - 1) / per;
    const dim3 grid((unsigned)(groups < GN_FWD_BLOCKS ? groups : GN_FWD_BLOCKS));
    if (first) hipLaunchKernelGGL((gated_norm_kernel<E, LPR, K, true>), grid, dim3(GN_THREADS), 0, st, p);
    else hipLaunchKernelGGL((gated_norm_kernel<E, LPR, K, false>), grid, dim3(GN_THREADS), 0, st, p);
  }
}

// Lanes per row and 16-byte units per lane, by the row's units: the fewest
// lanes that hold a row with one unit each, so that a wave takes several
// narrow rows, but eight at the least, which leaves lanes idle in rows of one
// to four units (2^21 rows of 8, 16, 32 bf16 values, both passes: 218, 246, 314 us;
// with one, two and four lanes 51, 94, 203 us).  From 65 to 128 units a wave takes
// two a lane, so that its sums need no LDS (2^15 rows of 1024 bf16 values: 133 us,
// with 256 lanes 142 us; of 512 fp32 values 88 and 100 us); beyond a workgroup's 256
// units a lane has several.
template <typename E>
void launch_e(const GatedNormParams &p, bool first, bool bwd, hipStream_t st) {
  const int u = p.D / Vec16<E>::N;
  if (u <= 8) launch_lk<E, 8, 1>(p, first, bwd, st);
  else if (u <= 16) launch_lk<E, 16, 1>(p, first, bwd, st);
  else if (u <= 32) launch_lk<E, 32, 1>(p, first, bwd, st);
  else if (u <= 64) launch_lk<E, 64, 1>(p, first, bwd, st);
  else if (u <= 128) launch_lk<E, 64, 2>(p, first, bwd, st);
  else if (u <= 256) launch_lk<E, 256, 1>(p, first, bwd, st);
  else if (u <= 512) launch_lk<E, 256, 2>(p, first, bwd, st);
  else if (u <= 1024) launch_lk<E, 256, 4>(p, first, bwd, st);
  else if constexpr (sizeof(E) == 4) launch_lk<E, 256, 8>(p, first, bwd, st);  // bf16 ends at 8192 / 8 units
}

}  // namespace
}  // namespace dn

using namespace dn;

extern "C" dn_status dn_gated_norm(int64_t rows, int32_t D, int32_t R, int32_t dtype, const void *x, const void *z,
                                   const float *w, float eps, int32_t gate_first, void *y, hipStream_t stream) {
  const dn_status st = check(rows, D, R, dtype, w);
  if (st != DN_OK) return st;
  if (rows == 0) return DN_OK;
  if (!x || !z || !y || !aligned16(x) || !aligned16(z) || !aligned16(y)) return DN_EINVAL;
  if (rows > INT32_MAX) return DN_EUNSUPPORTED;
  GatedNormParams p = {};
  p.x = x;
  p.z = z;
  p.w = w;
  p.y = y;
  p.rows = rows;
  p.D = D;
  p.R = R;
  p.eps = eps;
  if (dtype == DN_BF16) launch_e<bf16>(p, gate_first != 0, false, stream);
  else launch_e<float>(p, gate_first != 0, false, stream);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}

extern "C" size_t dn_gated_norm_bwd_workspace(int64_t rows, int32_t D, int32_t R) {
  if (rows < 0 || D <= 0 || R <= 0 || rows % R != 0) return 0;
  return 4 * (size_t)block_count(rows, R) * R * D;
}

extern "C" dn_status dn_gated_norm_bwd(int64_t rows, int32_t D, int32_t R, int32_t dtype, const void *x, const void *z,
                                       const float *w, float eps, int32_t gate_first, const void *dy, void *dx, void *dz,
                                       float *dw, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  const dn_status st = check(rows, D, R, dtype, w);
  if (st != DN_OK) return st;
  if (!dw) return DN_EINVAL;
  if (rows > 0 && (!x || !z || !dy || !dx || !dz)) return DN_EINVAL;
  for (const void *q : {x, z, dy, static_cast<const void *>(dx), static_cast<const void *>(dz)})
    if (!aligned16(q)) return DN_EINVAL;
  // a workgroup for every weight row at the least, and fewer than 2^32 threads
  if (rows > INT32_MAX || R >= 1 << 24) return DN_EUNSUPPORTED;
  if (!workspace || !aligned16(workspace) || workspace_bytes < dn_gated_norm_bwd_workspace(rows, D, R)) return DN_ENOWS;
  GatedNormParams p = {};
  p.x = x;
  p.z = z;
  p.dy = dy;
  p.w = w;
  p.dx = dx;
  p.dz = dz;
  p.dw = dw;
  p.part = static_cast<float *>(workspace);
  p.rows = rows;
  p.D = D;
  p.R = R;
  p.blocks = block_count(rows, R);
  p.eps = eps;
  if (dtype == DN_BF16) launch_e<bf16>(p, gate_first != 0, true, stream);
  else launch_e<float>(p, gate_first != 0, true, stream);
  if (hipGetLastError() != hipSuccess) return DN_EHIP;
  hipLaunchKernelGGL(gated_norm_sum_kernel, dim3(R, (D + SUM_COLS - 1) / SUM_COLS), dim3(GN_THREADS), 0, stream, p);
  return hipGetLastError() == hipSuccess ? DN_OK : DN_EHIP;
}
