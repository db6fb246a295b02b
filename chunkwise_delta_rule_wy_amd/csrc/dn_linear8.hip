// Product of 8-bit rows with 8-bit weights, with its epilogue, for gfx950:
//
//   y[m, n] = act(xs[m] ws[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n]
//
// x and w are 8-bit floats (4 exponent and 3 mantissa bits), act is none, silu
// or gelu, y is rounded to bf16 once.
//
// The products are the matrix instructions of 128 indices (16 x 16) and of 64
// (32 x 32); their rate is 4.4 to 4.5 PFLOP/s.  A lane gives them 32 bytes of one
// row; which of a block's indices these are is free, as long as x and w agree.  They
// align the products of eight neighbouring bytes to the largest one, cut 13 bits below
// its power of two, and add to fp32 sums: some 2e-4 of a sum of 4096 products, where
// y's rounding to bf16 gives 1.7e-3.  There is no fp32 y for that reason.  The 8-bit
// instruction of 16 indices cuts the same bits at half the rate (2.1 PFLOP/s), so that only
// conversions to bf16, with the rate of its instructions, would keep more.
// w is the left operand, so that a lane's results are consecutive columns n of
// one row m.
//
// Many rows: tiles of x and w pass through LDS, a block of 128 indices at a time,
// loaded directly (no registers) up to two blocks ahead.  A row of a tile is 128 bytes, half
// the span of the 64 banks; its 16-byte units are stored at unit ^ (row / 2 & 7), so
// that sixteen lanes reading one unit of sixteen rows meet all banks (with unit ^
// (row & 7), which only tells eight rows apart, every read took twice its time).
//
// 16384 x 8192 over 4096 indices take 422 to 438 us, 2.5 to 2.6 PFLOP/s at a clock that
// the power brings down to 1.9 GHz, with the matrix unit busy in 65 % of the cycles.
//
// Few rows: the weights are the traffic, and no tile of them is used twice; a
// workgroup takes 16 columns, and its waves share the indices and nothing else.
#include "dn.h"
#include "dn_internal.h"
#include "dn_wy.h"

namespace dn {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int BK = 128;  // indices (bytes of a row) of a tile

enum Act { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2 };

struct Linear8Params {
  const uint8_t *x, *w;
  const float *xs, *ws, *bias;  // bias may be null
  const bf16 *residual;         // may be null
  bf16 *y;
  int M, N, K;
  int act;
  int tm, tn;  // tiles over M and N
};

// what a lane reads instead of a row's indices behind K
__device__ const u128 g_zero16 = {{0, 0, 0, 0}};

__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.f + __expf(-z)); }
// z Phi(z), Phi(-|z|) = e^(-z^2 / 2) t Q(t) with t = 1 / (1 + 0.3677 |z|): Q is the
// polynomial of degree 6 that fits e^(z^2 / 2) Phi(-|z|) / t best (1.1e-6 of it for |z| up
// to 14), so that the value keeps its digits below zero too, where 1 + erf would lose them:
// with fp32's roundings 8e-6 of it, where y's rounding to bf16 gives 2e-3.  (1357 x 1001 over
// 2064 indices: 12.8 us, with erff 13.7, with no activation 11.6.)
__device__ __forceinline__ float gelu(float z) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.36769554f, 1.f));
  float q = __builtin_fmaf(t, 0.048311852f, -0.173576f);
  q = __builtin_fmaf(t, q, 0.15546185f);
  q = __builtin_fmaf(t, q, 0.040676955f);
  q = __builtin_fmaf(t, q, 0.13678895f);
  q = __builtin_fmaf(t, q, 0.14560027f);
  q = __builtin_fmaf(t, q, 0.14673667f);
  const float below = __builtin_amdgcn_exp2f(-0.7213475f * z * z) * t * q;
  return z * (z < 0.f ? below : 1.f - below);
}

// Tile of a workgroup.  Workgroups are dealt to the 8 XCDs round robin; each XCD gets a
// contiguous range of tiles, which run through bands of BAND rows of tiles, so that
// the tiles which are side by side in time share rows of x and of w in one L2
// (16384 x 8192 x 4096: 422 to 438 us; bands of 2 and 8 rows within that, and where the
// loads still set the pace 3 and 11 % longer).
constexpr int BAND = 4;
__device__ __forceinline__ void tile_of(const Linear8Params &p, int &tm, int &tn) {
  const int total = p.tm * p.tn, q = total >> 3, r = total & 7, xcd = blockIdx.x & 7;
  const int t = xcd * q + min(xcd, r) + (blockIdx.x >> 3);
  const int band = t / (BAND * p.tn), in = t - band * BAND * p.tn, high = min(BAND, p.tm - band * BAND);
  tm = band * BAND + in % high;
  tn = in / high;
}

// A 32-byte operand: the units `unit` (even) and unit + 1 of a row of a tile.
__device__ __forceinline__ i32x8 operand(uint32_t tile, int row, int unit) {
  const uint32_t at = tile + row * BK, swz = row >> 1 & 7;
  const i32x4 lo = wy::ld<i32x4>(at + ((unit ^ swz) << 4)), hi = wy::ld<i32x4>(at + (((unit + 1) ^ swz) << 4));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int TM, int TN, int WM, int WN, int RING, int ACT>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN)) void linear8_tile_kernel(Linear8Params p) {
  constexpr int WAVES = (TM / WM) * (TN / WN), STAGE = (TM + TN) * BK, NM = WM / 32, NN = WN / 32;
  __shared__ __attribute__((aligned(256))) char lds[RING * STAGE];
  __shared__ f32x2 cols[TN];  // (ws, bias) of a tile's columns
  const uint32_t base = (uint32_t)(size_t)(__attribute__((address_space(3))) char *)lds;
  const int lane = lane_id(), wave = wave_id();
  const int wm = (wave % (TM / WM)) * WM, wn = (wave / (TM / WM)) * WN;
  const int row = lane & 31, half = lane >> 5;
  const int blocks = (p.K + BK - 1) / BK, ragged = p.K % BK != 0;
  int tm, tn;
  tile_of(p, tm, tn);
  const int m0 = tm * TM, n0 = tn * TN;

  // A wave's share of a tile's rows, eight at a time: rows of w first, then of x.
  constexpr int PIECES = (TM + TN) / 8 / WAVES, OF_W = TN / 8 / WAVES;
  static_assert(PIECES * 8 * WAVES == TM + TN && OF_W * 8 * WAVES == TN, "the waves share the rows evenly");
  uint32_t src[PIECES];  // byte offsets from the tile's first row of w or x: K is at most 2^23
  // the unit that lands at lane % 8 of its row
  const auto unit = [&](int j) { return (lane & 7) ^ ((4 * (j * WAVES + wave) + (lane >> 4)) & 7); };
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    const int r = (j * WAVES + wave) * 8 + (lane >> 3);
    src[j] = (uint32_t)(j < OF_W ? min(r, p.N - 1 - n0) : min(r - TN, p.M - 1 - m0)) * (uint32_t)p.K + unit(j) * 16;
  }
  const uint8_t *w0 = p.w + (size_t)n0 * p.K, *x0 = p.x + (size_t)m0 * p.K;
  const auto load = [&](int j, int k, int stage, bool tail) {
    const uint8_t *from = (j < OF_W ? w0 : x0) + k;
    const uint32_t to = base + stage * STAGE + (j * WAVES + wave) * 1024;
    if (!tail) wy::dma16s(from, src[j], to);
    else wy::dma16(k + unit(j) * 16 < p.K ? (const void *)(from + src[j]) : (const void *)&g_zero16, to);
  };

  // The loop over K, a block of 128 indices a turn.  One wave has a SIMD to itself
  // in the large tiles, so that whatever it waits for stops the matrix unit.  Between
  // the products of the block's first half it reads the operands of the second,
  // whereupon the block's place is free (first barrier), and between those of the
  // second half it starts the loads of the block after the next, evenly spaced, as
  // bursts are slower.  The next block, whose loads were started a turn ago, is
  // waited for (second barrier) before the last quarter of the products, between
  // which its first operands are read.
  constexpr int PRODUCTS = NN * NM, OPERANDS = NN + NM, JOIN = PRODUCTS * 3 / 4;
  f32x16 acc[NN][NM];
  i32x8 f[2][OPERANDS];
  const auto read = [&](int set, int o, int stage) {
    const uint32_t at = base + stage * STAGE + (o < NN ? wn + 32 * o : TN + wm + 32 * (o - NN)) * BK;
    f[set][o] = operand(at, row, 4 * set + 2 * half);
  };
  const auto product = [&](int set, int i) {
    const int a = i / NM, b = i % NM;
    acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f[set][a], f[set][NN + b], acc[a][b], 0, 0, 0, 0, 0, 0);
  };
  // what a turn loads: the block after the next, that as the ragged last one, or
  // nothing; the last turn has no next block
  enum Mode { FULL, TAIL, NEXT, LAST };
  const auto turn = [&](auto mode_c, int k, int stage) {
    constexpr int mode = decltype(mode_c)::value;
#pragma unroll
    for (int i = 0; i < PRODUCTS; ++i) {
#pragma unroll
      for (int o = i * OPERANDS / PRODUCTS; o < (i + 1) * OPERANDS / PRODUCTS; ++o) read(1, o, stage);
      product(0, i);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < PRODUCTS; ++i) {
      if (mode <= TAIL && i == 0 && JOIN > 0) __syncthreads();
      if (mode != LAST && i == JOIN) {
        wy::wait_vm<mode == NEXT ? 0 : PIECES * JOIN / PRODUCTS>();
        __syncthreads();
      }
      if (mode != LAST && i >= JOIN) {
#pragma unroll
        for (int o = (i - JOIN) * OPERANDS / (PRODUCTS - JOIN); o < (i - JOIN + 1) * OPERANDS / (PRODUCTS - JOIN); ++o)
          read(0, o, stage ^ 1);
      }
      if (mode <= TAIL) {
#pragma unroll
        for (int j = i * PIECES / PRODUCTS; j < (i + 1) * PIECES / PRODUCTS; ++j)
          load(j, k + 2 * BK, stage, mode == TAIL);
      }
      product(1, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

#pragma unroll
  for (int j = 0; j < PIECES; ++j) load(j, 0, 0, p.K < BK);
  for (int n = threadIdx.x; n < TN; n += 64 * WAVES) {
    const int c = min(n0 + n, p.N - 1);
    cols[n] = (f32x2){p.ws[c], p.bias ? p.bias[c] : 0.f};
  }
  float xs[NM];
#pragma unroll
  for (int b = 0; b < NM; ++b) xs[b] = p.xs[min(m0 + wm + 32 * b + row, p.M - 1)];
#pragma unroll
  for (int a = 0; a < NN; ++a)
#pragma unroll
    for (int b = 0; b < NM; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.f;
  int at = 0, last;  // the last block's place
  if constexpr (RING == 2) {
    wy::wait_vm<0>();
    __syncthreads();
    if (blocks > 1) {
#pragma unroll
      for (int j = 0; j < PIECES; ++j) load(j, BK, 1, p.K < 2 * BK);
    }
#pragma unroll
    for (int o = 0; o < OPERANDS; ++o) read(0, o, 0);
    for (; at + 2 < blocks - ragged; ++at) turn(std::integral_constant<int, FULL>(), at * BK, at & 1);
    if (at + 2 < blocks) {
      turn(std::integral_constant<int, TAIL>(), at * BK, at & 1);
      ++at;
    }
    if (at + 1 < blocks) {
      turn(std::integral_constant<int, NEXT>(), at * BK, at & 1);
      ++at;
    }
    turn(std::integral_constant<int, LAST>(), at * BK, at & 1);
    last = at & 1;
  } else {
    // Small tiles: a block's products take far less than its loads, which are started
    // RING - 1 blocks ahead, and several workgroups of a CU fill each other's waits.
#pragma unroll
    for (int k = 1; k < RING - 1; ++k)
      if (k < blocks) {
#pragma unroll
        for (int j = 0; j < PIECES; ++j) load(j, k * BK, k, (k + 1) * BK > p.K);
      }
    for (int stage = 0; at < blocks; ++at) {
      if (at + RING - 2 < blocks) wy::wait_vm<(RING - 2) * PIECES>();
      else wy::wait_vm<0>();
      __syncthreads();
#pragma unroll
      for (int o = 0; o < OPERANDS; ++o) {
        read(0, o, stage);
        read(1, o, stage);
      }
      const int ahead = at + RING - 1, to = stage == 0 ? RING - 1 : stage - 1;  // the place of the block before
      if (ahead < blocks) {
        if ((ahead + 1) * BK <= p.K) {
#pragma unroll
          for (int j = 0; j < PIECES; ++j) load(j, ahead * BK, to, false);
        } else {
#pragma unroll
          for (int j = 0; j < PIECES; ++j) load(j, ahead * BK, to, true);
        }
      }
#pragma unroll
      for (int i = 0; i < PRODUCTS; ++i) {
        product(0, i);
        product(1, i);
      }
      last = stage;
      stage = stage == RING - 1 ? 0 : stage + 1;
    }
  }

  // Epilogue, in the place of the last block: ROUND times 32 rows m are finished
  // in the registers, where a lane has four neighbouring columns of one row, and
  // pass through the wave's own part of LDS as bf16, so that whole rows are
  // stored.  A residual comes into that place first, by direct loads.  16-byte
  // units of a row are stored at unit ^ swizzle(row).
  constexpr int PITCH = 2 * WN, UNITS = PITCH / 16, PART = STAGE / WAVES;
  constexpr int FIT = PART / (32 * PITCH), ROUND = FIT >= NM ? NM : FIT >= 2 ? 2 : FIT;
  static_assert(ROUND > 0 && NM % ROUND == 0, "a wave's part holds 32 rows at least");
  const uint32_t part = base + last * STAGE + wave * PART;
  const auto swizzle = [](int r) { return r / (256 / PITCH) % UNITS; };
  const int nw = n0 + wn;
  const bool whole = (p.N & 7) == 0;  // rows of y start at 16-byte units
  mfma_settle();
  __syncthreads();
#pragma unroll
  for (int b0 = 0; b0 < NM; b0 += ROUND) {
    const int mb = m0 + wm + 32 * b0;
    constexpr int STEP = 64 / UNITS;  // rows a pass
    const int u = lane % UNITS;
    if (p.residual && whole) {
#pragma unroll
      for (int r0 = 0; r0 < 32 * ROUND; r0 += STEP) {
        const int r = r0 + lane / UNITS, n = nw + 8 * (u ^ swizzle(r));
        wy::dma16(n < p.N ? (const void *)(p.residual + (size_t)min(mb + r, p.M - 1) * p.N + n) : (const void *)&g_zero16,
                  part + r0 * PITCH);
      }
      wy::wait_vm<0>();
      asm volatile("" ::: "memory");  // no read of that place before the wait
    }
#pragma unroll
    for (int a = 0; a < NN; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 32 * a + 8 * i + 4 * half;
        const f32x4 c01 = *reinterpret_cast<const f32x4 *>(&cols[wn + n]);
        const f32x4 c23 = *reinterpret_cast<const f32x4 *>(&cols[wn + n + 2]);
#pragma unroll
        for (int b = b0; b < b0 + ROUND; ++b) {
          const int r = 32 * (b - b0) + row;
          const uint32_t to = part + r * PITCH + (((n >> 3) ^ swizzle(r)) << 4) + 8 * half;
          float v[4];
          v[0] = __builtin_fmaf(acc[a][b][4 * i] * xs[b], c01[0], c01[1]);
          v[1] = __builtin_fmaf(acc[a][b][4 * i + 1] * xs[b], c01[2], c01[3]);
          v[2] = __builtin_fmaf(acc[a][b][4 * i + 2] * xs[b], c23[0], c23[1]);
          v[3] = __builtin_fmaf(acc[a][b][4 * i + 3] * xs[b], c23[2], c23[3]);
          if (ACT == ACT_SILU) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = silu(v[e]);
          } else if (ACT == ACT_GELU) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = gelu(v[e]);
          }
          if (p.residual) {
            bf16x4 res;
            if (whole) {
              res = wy::ld<bf16x4>(to);
            } else {
              const bf16 *from = p.residual + (size_t)min(m0 + wm + 32 * b + row, p.M - 1) * p.N;
#pragma unroll
              for (int e = 0; e < 4; ++e) res[e] = from[min(nw + n + e, p.N - 1)];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += to_f<bf16>(res[e]);
          }
          wy::st<u32x2>(to, (u32x2){pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])});
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    wave_lds_fence();
    if (whole) {
#pragma unroll 4
      for (int r0 = 0; r0 < 32 * ROUND; r0 += STEP) {
        const int r = r0 + lane / UNITS, m = mb + r, n = nw + 8 * u;
        const u32x4 v = wy::ld<u32x4>(part + r * PITCH + ((u ^ swizzle(r)) << 4));
        if (m < p.M && n < p.N) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p.y + (size_t)m * p.N + n));
      }
    } else {  // one column a lane
#pragma unroll 4
      for (int o = lane; o < 32 * ROUND * WN; o += 64) {
        const int r = o / WN, n = o % WN;
        const bf16 v = wy::ld<bf16>(part + r * PITCH + (((n >> 3) ^ swizzle(r)) << 4) + 2 * (n & 7));
        if (mb + r < p.M && nw + n < p.N) p.y[(size_t)(mb + r) * p.N + nw + n] = v;
      }
    }
    wave_lds_fence();
  }
}

// Few rows: 16 columns a workgroup, whose waves take a contiguous part of the indices
// each, in blocks of 128.  The blocks pass through the wave's own part of LDS, two
// at a time and without barriers, as in the tiles: a load into registers would touch
// 16 rows at once, which takes twice the time for the same bytes (64 x 4096 x 4096:
// 12.3 us, so 8.3).  What is left: the launch, four blocks a wave that depend on nothing
// but arrive one after the other, the exchange of the waves' sums, and with many rows x,
// which every workgroup reads whole (64 rows of 4096: 256 KB beside 64 KB of weights, from
// the L2's).
constexpr int FEW_WAVES = 8;

template <int MT>
__global__ __launch_bounds__(64 * FEW_WAVES) void linear8_few_kernel(Linear8Params p) {
  constexpr int BLOCK = 16 * (1 + MT) * BK, PIECES = 2 * (1 + MT);
  constexpr int PART = FEW_WAVES * 16 * MT * 20 * 4, LDS = 2 * FEW_WAVES * BLOCK > PART ? 2 * FEW_WAVES * BLOCK : PART;
  __shared__ __attribute__((aligned(256))) char lds[LDS];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id()), row = lane & 15, unit = 2 * (lane >> 4);
  const uint32_t base = (uint32_t)(size_t)(__attribute__((address_space(3))) char *)lds + wave * 2 * BLOCK;
  const int n0 = blockIdx.x * 16;
  // eight rows a piece: two pieces of w, then those of x
  uint32_t src[PIECES];
  const uint8_t *w0 = p.w + (size_t)n0 * p.K;
  const auto from = [&](int j) { return (lane & 7) ^ ((4 * j + (lane >> 4)) & 7); };  // the unit that lands at lane % 8
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    const int r = 8 * j + (lane >> 3);
    src[j] = (uint32_t)(j < 2 ? min(r, p.N - 1 - n0) : min(r - 16, p.M - 1)) * (uint32_t)p.K + from(j) * 16;
  }
  const auto load = [&](int k, int stage) {
    const bool whole = k + BK <= p.K;
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const uint8_t *at = (j < 2 ? w0 : p.x) + k;
      const uint32_t to = base + stage * BLOCK + j * 1024;
      if (whole) wy::dma16s(at, src[j], to);
      else wy::dma16(k + from(j) * 16 < p.K ? (const void *)(at + src[j]) : (const void *)&g_zero16, to);
    }
  };
  const int blocks = (p.K + BK - 1) / BK, per = (blocks + FEW_WAVES - 1) / FEW_WAVES;
  const int first = wave * per, end = min(first + per, blocks);
  f32x4 acc[MT];
#pragma unroll
  for (int b = 0; b < MT; ++b) acc[b] = zero4();
  if (first < end) load(first * BK, 0);
  if (first + 1 < end) load((first + 1) * BK, 1);
  for (int t = first; t < end; ++t) {
    if (t + 1 < end) wy::wait_vm<PIECES>();
    else wy::wait_vm<0>();
    asm volatile("" ::: "memory");  // no read before the wait
    const uint32_t at = base + ((t - first) & 1) * BLOCK;
    const i32x8 fw = operand(at, row, unit);
    i32x8 fx[MT];
#pragma unroll
    for (int b = 0; b < MT; ++b) fx[b] = operand(at + 16 * BK, 16 * b + row, unit);
    wave_lds_fence();
    if (t + 2 < end) load((t + 2) * BK, (t - first) & 1);
#pragma unroll
    for (int b = 0; b < MT; ++b)
      acc[b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fx[b], acc[b], 0, 0, 0, 0, 0, 0);
  }
  mfma_settle();
  __syncthreads();
  float (*part)[16 * MT][20] = reinterpret_cast<float (*)[16 * MT][20]>(lds);
#pragma unroll
  for (int b = 0; b < MT; ++b) *reinterpret_cast<f32x4 *>(&part[wave][16 * b + row][4 * (lane >> 4)]) = acc[b];
  __syncthreads();
  for (int o = threadIdx.x; o < 256 * MT; o += 64 * FEW_WAVES) {
    const int m = o >> 4, n = o & 15;
    if (m >= p.M || n0 + n >= p.N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < FEW_WAVES; ++k) s += part[k][m][n];
    s = s * p.xs[m] * p.ws[n0 + n] + (p.bias ? p.bias[n0 + n] : 0.f);
    if (p.act == ACT_SILU) s = silu(s);
    else if (p.act == ACT_GELU) s = gelu(s);
    const size_t at = (size_t)m * p.N + n0 + n;
    if (p.residual) s += to_f<bf16>(p.residual[at]);
    p.y[at] = to_e<bf16>(s);
  }
}

// ------------------------------------------------------------------- host

template <int TM, int TN, int WM, int WN, int RING>
hipError_t launch_tile(Linear8Params &p, hipStream_t st) {
  p.tm = (p.M + TM - 1) / TM;
  p.tn = (p.N + TN - 1) / TN;
  const int64_t tiles = (int64_t)p.tm * p.tn;
  const dim3 grid((unsigned)tiles), thr(64 * (TM / WM) * (TN / WN));
  if (p.act == ACT_SILU) hipLaunchKernelGGL((linear8_tile_kernel<TM, TN, WM, WN, RING, ACT_SILU>), grid, thr, 0, st, p);
  else if (p.act == ACT_GELU) hipLaunchKernelGGL((linear8_tile_kernel<TM, TN, WM, WN, RING, ACT_GELU>), grid, thr, 0, st, p);
  else hipLaunchKernelGGL((linear8_tile_kernel<TM, TN, WM, WN, RING, ACT_NONE>), grid, thr, 0, st, p);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_few(const Linear8Params &p, hipStream_t st) {
  hipLaunchKernelGGL(linear8_few_kernel<MT>, dim3((unsigned)((p.N + 15) / 16)), dim3(64 * FEW_WAVES), 0, st, p);
  return hipGetLastError();
}

// The tiles by their measured times: `first` for up to 256 of them, one for each CU, and
// `more` for every 256 beyond (tenths of us over 4096 indices).
int64_t cost(const Linear8Params &p, int t, int first, int more) {
  const int64_t n = (int64_t)((p.M + t - 1) / t) * ((p.N + t - 1) / t), rounds = (n + 255) / 256;
  return rounds <= 1 ? first : more * rounds;
}

hipError_t launch(Linear8Params &p, hipStream_t st) {
  // Few rows, of which a CU holds two workgroups (up to 16 rows) or one: up to two rounds
  // of these, or one where 64 rows make it longer, and tiles beyond.  In us, few [tiles]: over
  // 4096 indices 64 rows of 4096 columns 8.4 [11.0], of 6144 15.0 [13.9], of 16384 26.8
  // [15.7]; 32 of 4096 6.4 [10.9], of 8192 12.8 [13.6], of 12288 17.9 [16.0]; 1 of 4096 5.1
  // [10.8], of 16384 13.7 [13.8], of 65536 45.0 [45.7]; over 1024, 1 of 16384 5.7 [6.0], of
  // 65536 17.6 [15.0].
  const int64_t few = ((int64_t)p.N + 15) / 16;
  if (p.M <= 16 && few <= 1024) return launch_few<1>(p, st);
  if (p.M > 16 && p.M <= 32 && few <= 512) return launch_few<2>(p, st);
  if (p.M > 32 && p.M <= 64 && few <= 256) return launch_few<4>(p, st);
  // In us over 4096 indices with tiles of 64, 128 and 256: 256 x 4096 12.6, 17.9, 43.6; 768 x
  // 4096 24.8, 20.2, 44.3; 3000 x 4096 81.8, 50.4, 52.1; 4096 x 4096 118, 65.6, 56.8; 4096 x 4097
  // 126, 83.6, 126.
  const int64_t small = cost(p, 64, 126, 70), medium = cost(p, 128, 190, 165), large = cost(p, 256, 560, 560);
  if (large <= medium && large <= small) return launch_tile<256, 256, 128, 128, 2>(p, st);
  if (medium <= small) return launch_tile<128, 128, 64, 64, 2>(p, st);
  return launch_tile<64, 64, 32, 32, 4>(p, st);
}

}  // namespace
}  // namespace dn

using namespace dn;

extern "C" dn_status dn_linear8(int32_t M, int32_t N, int32_t K, const void *x, const float *xs, const void *w,
                                const float *ws, const float *bias, const void *residual, int32_t act, void *y,
                                hipStream_t stream) {
  if (M < 0 || N <= 0 || K <= 0 || act < ACT_NONE || act > ACT_GELU) return DN_EINVAL;
  // the rows' 16-byte units, a tile's 32-bit byte offsets, and a grid's threads (fewer than 2^32)
  if (K % 16 != 0 || K > 1 << 23) return DN_EUNSUPPORTED;
  if (((int64_t)M + 63) / 64 * (((int64_t)N + 63) / 64) > UINT32_MAX / 256 || N > 1 << 26 || M > INT32_MAX - 256)
    return DN_EUNSUPPORTED;
  if (M == 0) return DN_OK;
  if (!x || !xs || !w || !ws || !y) return DN_EINVAL;
  for (const void *q : {x, w, residual, static_cast<const void *>(y)})
    if (reinterpret_cast<uintptr_t>(q) & 15u) return DN_EINVAL;
  Linear8Params p = {};
  p.x = static_cast<const uint8_t *>(x);
  p.w = static_cast<const uint8_t *>(w);
  p.xs = xs;
  p.ws = ws;
  p.bias = bias;
  p.residual = static_cast<const bf16 *>(residual);
  p.y = static_cast<bf16 *>(y);
  p.M = M;
  p.N = N;
  p.K = K;
  p.act = act;
  return launch(p, stream) == hipSuccess ? DN_OK : DN_EHIP;
}
