// One token of the selective state space scan per (batch, head):
//
//   h' = exp(s A) h + s k v^T,   o = h'^T q + skip v      (s = softplus(dt + dt_bias))
//
// The state is read and written once and nothing else weighs against it, so
// the kernel is bound by HBM: a workgroup streams a COLS-wide slice of one
// state, every thread keeping four columns of Dk / RG rows in registers
// between load and store, all loads issued before the first use.  256
// sequences, 32 heads of 128 x 128: 1.08 GB in 207 us, 5.2 TB/s, the rate of a
// large copy.  A single sequence is bound by the call and the launch (9 us).
#include "dn_ssm.h"

namespace dn {
namespace {

template <typename E, int DK, int COLS>
__global__ __launch_bounds__(NTHR) void ssm_step_kernel(SsmStepParams p) {
  constexpr int CG = COLS / 4, RG = NTHR / CG, RPT = DK / RG;
  __shared__ float s_o[RG][COLS];
  const int nsl = p.DV / COLS;
  const int bh = blockIdx.x / nsl, sl = blockIdx.x % nsl;
  const int b = bh / p.H, h = bh % p.H;
  const int t = threadIdx.x, cg = t % CG, rg = t / CG;
  const int c0 = sl * COLS + 4 * cg;
  const size_t qk = ((size_t)b * p.G + h / (p.H / p.G)) * DK;
  const E *q = static_cast<const E *>(p.q) + qk, *k = static_cast<const E *>(p.k) + qk;
  const E *v = static_cast<const E *>(p.v) + (size_t)bh * p.DV + c0;
  float *st = p.state + (size_t)bh * DK * p.DV + c0;
  f32x4 hv[RPT];
  float qr[RPT], kr[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) hv[i] = *reinterpret_cast<const f32x4 *>(st + (size_t)(rg + RG * i) * p.DV);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    qr[i] = to_f<E>(q[rg + RG * i]);
    kr[i] = to_f<E>(k[rg + RG * i]);
  }
  const float s = softplus(p.dt[bh] + (p.bias ? p.bias[h] : 0.f));
  const float alpha = __expf(s * p.A[h]);
  f32x4 vv;
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = to_f<E>(v[e]);
  const f32x4 sv = s * vv;
  f32x4 o = zero4();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    hv[i] = alpha * hv[i] + kr[i] * sv;
    o += qr[i] * hv[i];
    *reinterpret_cast<f32x4 *>(st + (size_t)(rg + RG * i) * p.DV) = hv[i];
  }
  *reinterpret_cast<f32x4 *>(&s_o[rg][4 * cg]) = o;
  __syncthreads();
  if (t < CG) {
    f32x4 sum = zero4();
#pragma unroll
    for (int r = 0; r < RG; ++r) sum += *reinterpret_cast<const f32x4 *>(&s_o[r][4 * t]);
    const float skip = p.skip ? p.skip[h] : 0.f;
    E *out = static_cast<E *>(p.o) + (size_t)bh * p.DV + c0;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = to_e<E>(sum[e] + skip * vv[e]);
  }
}

template <typename E>
void launch(const SsmStepParams &p, int DK, hipStream_t stream) {
  // 128-wide slices where Dv has them, else 64
  const bool wide = p.DV % 128 == 0;
  const dim3 grid((unsigned)((int64_t)p.B * p.H * (p.DV / (wide ? 128 : 64))));
  if (DK == 64) {
    if (wide) hipLaunchKernelGGL((ssm_step_kernel<E, 64, 128>), grid, dim3(NTHR), 0, stream, p);
    else hipLaunchKernelGGL((ssm_step_kernel<E, 64, 64>), grid, dim3(NTHR), 0, stream, p);
  } else {
    if (wide) hipLaunchKernelGGL((ssm_step_kernel<E, 128, 128>), grid, dim3(NTHR), 0, stream, p);
    else hipLaunchKernelGGL((ssm_step_kernel<E, 128, 64>), grid, dim3(NTHR), 0, stream, p);
  }
}

}  // namespace

hipError_t launch_ssm_step(const SsmStepParams &p, int dtype, int DK, hipStream_t stream) {
  if (dtype == 1) launch<bf16>(p, DK, stream);
  else launch<float>(p, DK, stream);
  return hipGetLastError();
}

}  // namespace dn
