// Shared parts of the selective state space scan's kernels (gfx950).
//
// Per sequence and head (q, k shared by the H / G heads of a group):
//
//   s_t = softplus(dt_t + dt_bias),  a_t = s_t A
//   h_t = exp(a_t) h_{t-1} + s_t k_t v_t^T      (h = S^T, Dk x Dv)
//   o_t = h_t^T q_t + skip v_t
//
// Over a chunk of 64 tokens, with b = cumsum a, gamma = exp b,
// Gamma_rj = exp(b_r - b_j) for j <= r and w_j = exp(b_63 - b_j):
//
//   O  = ((Q K^T) * Gamma) diag(s) V + diag(gamma) Q h + skip V
//   h+ = gamma_63 h + K^T diag(w s) V
//
// and going back, with dh+ the gradient of the chunk's end state,
//
//   dh = gamma_63 dh+ + Q^T diag(gamma) dO.
//
// Both are the same sweep S <- gamma_63 S + X^T diag(c) Y, over (k, v, w s)
// forwards and (q, dO, gamma) backwards.  A sequence is cut into segments of
// whole chunks, so that few long sequences still fill the device: one sweep
// from a zero state leaves each segment's own end state, an elementwise pass
// joins them to the segments' start states, and the segments then run side by
// side.
//
// Precision.  k, v, q and dO are bf16 and enter the matrix products exactly.
// Everything that feeds a state or an fp32 gradient is an fp32 value split
// into three bf16 parts (split3: 24 bits), one product each, so that states,
// ddt and the parameter gradients keep fp32 accuracy; what feeds only bf16
// outputs is rounded to bf16 once.  Log decays are summed in double and used
// as differences, so that neither long chunks nor strong decays lose the
// ratio of two neighbours.
#pragma once

#include "dn_chunk.h"
#include "dn_wy.h"

namespace dn {

constexpr int SSM_TILE = 64;  // Dv columns of a workgroup

// A workgroup of the sweeps and the forward pass takes 64 columns, or twice 64
// that share their keys: two column tiles of one head where Dv is a multiple
// of 128, else tiles of two heads of one group where it has an even number.
// Keys and queries are then loaded, and their fragments read from LDS, once for
// both.
enum SsmPair { SSM_SINGLE = 0, SSM_TILES = 1, SSM_HEADS = 2 };

struct SsmParams {
  const bf16 *q, *k, *v, *dO;
  const float *dt, *A, *bias, *skip;  // bias, skip may be null
  const float *h0, *dhT;              // may be null
  const int32_t *cu;                  // packed sequences, or null
  const int32_t *seg_base, *seg_seq;      // packed and cut: segment table
  const int32_t *chunk_base, *chunk_seq;  // packed: chunk table (backward)
  bf16 *o;
  float *hT;                 // may be null
  float *seg_state[2];       // per segment and head: own end state, then start state (0 forwards, 1 backwards)
  double *seg_decay;         // per segment and head: sum of the log2 decays
  float *states, *dstates;   // backward: state entering each chunk, gradient of the state leaving it
  bf16 *dq, *dk, *dv;
  float *dq_part, *dk_part;  // fp32 partial sums over sets of heads, or null
  float *ddt, *dA, *ddt_bias, *dskip, *dh0;  // ddt_bias, dskip, dh0 may be null
  double *par_part;          // [chunk][H][3]: dA, ddt_bias, dskip
  int64_t rows;              // B T
  int T, H, G, DV, N;
  int ntiles;                // Dv / 64
  int pair;                  // columns of a workgroup: see SsmPair
  int split;                 // segments are joined through seg_state
  int NS, segc;              // segments of a sequence (not packed), chunks of a segment
  int NC;                    // chunks of a sequence (not packed)
  int nseg, nchunks;         // upper bounds over all sequences
  int sets, set_heads;       // backward: sets of heads of a group, heads of a set
  int zero_tail;             // packed: clear the results' rows behind the last sequence
};

hipError_t launch_ssm_sweep(const SsmParams &p, int DK, bool store, bool backward, hipStream_t stream);
hipError_t launch_ssm_join(const SsmParams &p, int DK, bool backward, hipStream_t stream);
hipError_t launch_ssm_fwd(const SsmParams &p, int DK, hipStream_t stream);
hipError_t launch_ssm_grad(const SsmParams &p, int DK, hipStream_t stream);

struct SsmStepParams {
  const void *q, *k, *v;
  const float *dt, *A, *bias, *skip;
  float *state;
  void *o;
  int B, H, G, DV;
};
hipError_t launch_ssm_step(const SsmStepParams &p, int dtype, int DK, hipStream_t stream);

// Workgroups are dealt to the 8 XCDs round robin; this gives each XCD (one L2)
// a contiguous range of the work items, so that the heads that share a
// segment's keys and queries meet in one L2.
__device__ __forceinline__ int xcd_item(int x, int total) {
  const int q = total >> 3, r = total & 7, xcd = x & 7;
  return xcd * q + min(xcd, r) + (x >> 3);
}

// A segment: sequence n, first token row, tokens, place in the sequence.  Where
// sequences are not cut, every sequence is one segment, also one without
// tokens.
struct Segment {
  int n, len, chunk;  // chunk: its first chunk within the sequence
  size_t row;
  bool first, last;
};
__device__ __forceinline__ bool segment(const SsmParams &p, int seg, Segment &s) {
  int start, len;
  if (p.cu) {
    s.n = p.split ? p.seg_seq[seg] : seg;
    if (s.n < 0) return false;
    const int i = p.split ? seg - p.seg_base[s.n] : 0, t0 = p.cu[s.n];
    len = p.cu[s.n + 1] - t0;
    s.chunk = i * p.segc;
    start = s.chunk * CH;
    s.row = (size_t)t0 + start;
  } else {
    s.n = seg / p.NS;
    len = p.T;
    s.chunk = (seg - s.n * p.NS) * p.segc;
    start = s.chunk * CH;
    s.row = (size_t)s.n * p.T + start;
  }
  s.first = start == 0;
  s.last = len - start <= p.segc * CH;
  s.len = s.last ? len - start : p.segc * CH;
  return true;
}
// Clears the rows behind the last packed sequence of a result with rows of
// `units` elements of T, all workgroups together.
template <typename T>
__device__ __forceinline__ void clear_tail(const SsmParams &p, void *result, int64_t units) {
  T *out = static_cast<T *>(result);
  const int64_t end = p.rows * units;
  for (int64_t i = p.cu[p.N] * units + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < end;
       i += (int64_t)gridDim.x * blockDim.x)
    out[i] = T{};
}
// its first chunk's number among all
__device__ __forceinline__ int first_chunk(const SsmParams &p, const Segment &s) {
  return (p.cu ? p.chunk_base[s.n] : s.n * p.NC) + s.chunk;
}

// A chunk's states lie in the workspace as the sweeps hold them: units of four
// columns, in the order [block of 16 columns][block of 16 Dk rows][row][unit],
// so that a wave's store is 1 KiB in one piece (4 x 4096 tokens, 32 heads, 128 x
// 64: the storing sweeps took 140 us and the gradient kernel, which reads them
// and has become faster since, 250 us; with rows of Dv columns 178 and 270 us).
// The byte offset of a unit.
template <int DK>
__device__ __forceinline__ uint32_t chunk_state_unit(int t, int c, int m, int u) {
  return 16 * (((c * (DK / 16) + t) * 16 + m) * 4 + u);
}

// e^x for -200 <= x <= 0: 2^n e^r, x = n ln 2 + r with ln 2 in two parts (the
// first has 16 bits, so that its product with n is exact), e^r by its series
// up to r^7 / 7! (|r| < 0.35: the rest is below 2^-25 of r).
__device__ __forceinline__ float exp_of(float x) {
  const float n = __builtin_rintf(x * wy::LOG2E);
  float r = __builtin_fmaf(n, -0.693145751953125f, x);
  r = __builtin_fmaf(n, -1.428606765330187e-06f, r);
  float p = 1.f / 5040;
  p = __builtin_fmaf(p, r, 1.f / 720);
  p = __builtin_fmaf(p, r, 1.f / 120);
  p = __builtin_fmaf(p, r, 1.f / 24);
  p = __builtin_fmaf(p, r, 1.f / 6);
  p = __builtin_fmaf(p, r, 0.5f);
  return __builtin_ldexpf(1.f + __builtin_fmaf(p * r, r, r), (int)n);
}
// log(1 + e^x) = max(x, 0) + log1p(y), y = e^-|x|; log1p(y) = 2 atanh z with z =
// y / (2 + y) <= 1/3, by the series 2 (z + z^3 / 3 + ...  + z^15 / 15).  The
// quotient is corrected for its own rounding and for that of 2 + y.  A step size
// is off by 4e-8 on average and without a bias (below 1e-8 of it): one that all
// tokens share does not cancel in dA as the tokens' terms may.  The largest
// negative steps, minus infinity among them, give 0; NaN stays NaN.
__device__ __forceinline__ float softplus(float x) {
  const float n = -fabsf(x);
  const float y = exp_of(n < -200.f ? -200.f : n), d = 2.f + y, e = y - (d - 2.f);
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
  float z = y * r;
  z = __builtin_fmaf(__builtin_fmaf(-e, z, __builtin_fmaf(-d, z, y)), r, z);
  const float q = z * z;
  float s = 1.f / 15;
  s = __builtin_fmaf(s, q, 1.f / 13);
  s = __builtin_fmaf(s, q, 1.f / 11);
  s = __builtin_fmaf(s, q, 1.f / 9);
  s = __builtin_fmaf(s, q, 1.f / 7);
  s = __builtin_fmaf(s, q, 1.f / 5);
  s = __builtin_fmaf(s, q, 1.f / 3);
  z += z;
  return (x < 0.f ? 0.f : x) + __builtin_fmaf(z * q, s, z);
}

// The step of lane l's token of a chunk of L > 0 tokens, before bias and
// softplus; lanes from L on repeat the last token.  Loaded ahead of its use, with
// nothing computed from it there: that would wait for it, and for all loads
// before it.
__device__ __forceinline__ float load_step(const SsmParams &p, size_t row0, int L, int h) {
  return p.dt[(row0 + min(lane_id(), L - 1)) * p.H + h];
}

// inclusive prefix sum over the 64 lanes of a wave, in double
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp0d(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_incl_scan_d(double x) {
  x += dpp0d<0x111>(x);
  x += dpp0d<0x112>(x);
  x += dpp0d<0x114>(x);
  x += dpp0d<0x118>(x);
  x += dpp0d<0x142, 0xa>(x);
  x += dpp0d<0x143, 0xc>(x);
  return x;
}
// sum over the 16 lanes of each row
__device__ __forceinline__ double row_sum16_d(double x) {
  x += dpp0d<0xB1>(x);
  x += dpp0d<0x4E>(x);
  x += dpp0d<0x124>(x);
  x += dpp0d<0x128>(x);
  return x;
}
// over the four rows of 16 lanes: the sum, and the sum of the rows after this one
__device__ __forceinline__ float row_suffix(float x, int g, float &after) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float pair = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(pair), __float_as_uint(pair), false, false);
  const float hi = __uint_as_float(b[1]);
  after = (g & 1 ? 0.f : __uint_as_float(a[1])) + (g & 2 ? 0.f : hi);
  return __uint_as_float(b[0]) + hi;
}
// sums over the four rows of 16 lanes of N = 2 or 4 values at once: row g gets
// that of x[g % N]
template <int N>
__device__ __forceinline__ float rows_sums(const float (&x)[N]) {
  static_assert(N == 2 || N == 4, "a value for every row, or for every other");
  auto halves = [](float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const float a = halves(x[0], x[N - 2]), b = halves(x[1], x[N - 1]);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// sums over the 16 lanes of a row of four values at once: lane m gets that of x[m % 4]
__device__ __forceinline__ float row_sums16(const f32x4 &x, int m) {
  const bool b0 = m & 1, b1 = m & 2;
  const float a = (b0 ? x[1] : x[0]) + dpp0<0xB1>(b0 ? x[0] : x[1]);
  const float b = (b0 ? x[3] : x[2]) + dpp0<0xB1>(b0 ? x[2] : x[3]);
  float c = (b1 ? b : a) + dpp0<0x4E>(b1 ? a : b);
  c += dpp0<0x124>(c);
  return c + dpp0<0x128>(c);
}
__device__ __forceinline__ double lane_val_d(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Gate table of one (chunk, head): s, the log2 decays b = bh + bl (two floats
// hold them to 2^-48), gamma, w, w s; `last` = gamma_63.
struct GateTab {
  alignas(256) float s[CH];
  float bh[CH], bl[CH], gam[CH], w[CH], ws[CH];
  float last, A, skip, pad;  // A and skip: the gradient kernel's
};
// One wave fills the table from the raw step sizes of its lanes' tokens (lanes
// from L on are padding: no decay, no input, gamma 0).  Returns the chunk's log2 decay.
__device__ __forceinline__ double fill_gates(GateTab &t, float raw, float A, int L) {
  const int l = lane_id();
  const float s = l < L ? softplus(raw) : 0.f;
  // a decay past 1e30 is zero as well, and sums of 64 stay within the floats' range
  const double a = (double)s * ((double)A * 1.4426950408889634074);
  const double b = wave_incl_scan_d(a < -1e30 ? -1e30 : a);
  const double total = lane_val_d(b, 63);
  const float bh = (float)b, bl = (float)(b - (double)bh);
  const float w = wy::fexp2((float)(total - b));
  t.s[l] = s;
  t.bh[l] = bh;
  t.bl[l] = bl;
  t.gam[l] = l < L ? wy::fexp2(bh) * (1.f + 0.6931471806f * bl) : 0.f;
  t.w[l] = w;
  t.ws[l] = w * s;
  if (l == 0) {
    const float th = (float)total;
    t.last = wy::fexp2(th) * (1.f + 0.6931471806f * (float)(total - (double)th));
  }
  return total;
}
__device__ __forceinline__ f32x4 lds4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
// Keeps a value's computation where it stands: without it a select between
// the value and zero becomes a branch around the computation, one for each
// element.
__device__ __forceinline__ float computed(float x) {
  asm("" : "+v"(x));
  return x;
}
// A lane-dependent value that the compiler takes for a new one here: what is
// computed from it is computed where it is used, instead of being held in
// registers (or spilled) across a loop that needs them all.
template <typename T>
__device__ __forceinline__ T fresh(T x) {
  asm volatile("" : "+v"(x));
  return x;
}
// The decay ratios Gamma of four rows r = r0 .. r0 + 3 to one column, or of one
// row to four columns j = r0 .. (sign -1), from the table's entries; ratios
// whose row is before their column come out as anything.
__device__ __forceinline__ f32x4 decay_ratios(const GateTab &t, int r0, float bh, float bl, float sign) {
  const f32x4 h = lds4(t.bh + r0), l = lds4(t.bl + r0);
  f32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = wy::fexp2(sign * ((h[i] - bh) + (l[i] - bl)));
  return x;
}

// x = p0 + p1 + p2 to 24 bits, each part a bf16 operand fragment
struct Split {
  bf16x8 p[3];
};
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ Split split3(const float (&x)[8]) {
  Split r;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = pk_bf16(v[2 * i], v[2 * i + 1]);
      if (k < 2) {
        v[2 * i] -= bf_lo(u[i]);
        v[2 * i + 1] -= bf_hi(u[i]);
      }
    }
    r.p[k] = __builtin_bit_cast(bf16x8, u);
  }
  return r;
}
// the eight elements of a bf16 fragment as floats
__device__ __forceinline__ void unpack8(const bf16x8 &f, float (&x)[8]) {
  const u32x4 u = __builtin_bit_cast(u32x4, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf_lo(u[i]);
    x[2 * i + 1] = bf_hi(u[i]);
  }
}

// the wave's number, as the scalar that it is
__device__ __forceinline__ int wave_number() { return __builtin_amdgcn_readfirstlane(wave_id()); }

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// An LDS matrix of COLS bf16 columns (64 or 128) without padding; the 16-byte
// unit u of row r sits at unit position u ^ f(r).  With f below, 16 rows of one
// unit (16-byte row reads), 32 lanes of half units (8-byte row reads) and the
// four rows by two units of a transposed read all fall into different banks.
template <int COLS>
struct Swz {
  static_assert(COLS == 64 || COLS == 128, "rows of 8 or 16 units");
  static constexpr int RB = 2 * COLS;  // bytes of a row
  __device__ static __forceinline__ int f(int r) {
    return COLS == 128 ? ((r & 3) << 2 | ((r >> 2) & 3)) : ((r & 2) << 1 | ((r >> 2) & 3));
  }
  // byte offset of unit u of row r
  __device__ static __forceinline__ uint32_t off(int r, int u) { return r * RB + ((u ^ f(r)) << 4); }
  // A lane's address within a tile is one base XOR a constant of the column
  // block plus an immediate offset of the row block (matrices start at multiples
  // of 256 bytes, and f repeats every 16 rows).
  //
  // 32-index fragments of rows 16 t + m, columns 32 kb + 8 g .. + 7
  __device__ static __forceinline__ uint32_t row_base(uint32_t base, int l) { return base + off(l & 15, l >> 4); }
  __device__ static __forceinline__ bf16x8 row(uint32_t b, int t, int kb) {
    return wy::ld<bf16x8>((b ^ (64 * kb)) + 16 * RB * t);
  }
  // four columns 16 c + 4 g .. + 3 of rows 16 t + m
  __device__ static __forceinline__ uint32_t quad_base(uint32_t base, int l) {
    return base + off(l & 15, l >> 5) + 8 * ((l >> 4) & 1);
  }
  __device__ static __forceinline__ uint32_t quad(uint32_t b, int t, int c) { return (b ^ (32 * c)) + 16 * RB * t; }
  // rows 16 t + m, columns 32 kb + 4 g .. + 3 and 32 kb + 16 + 4 g .. + 3: the
  // order of two stacked accumulator tiles
  __device__ static __forceinline__ bf16x8 row_stacked(uint32_t quad_b, int t, int kb) {
    return wy::cat(wy::ld<bf16x4>(quad(quad_b, t, 2 * kb)), wy::ld<bf16x4>(quad(quad_b, t, 2 * kb + 1)));
  }
  // transposed: columns 16 c + m, contraction over the rows 32 kb + 8 g .. + 7
  struct Col {
    uint32_t a, b;
  };
  __device__ static __forceinline__ Col col_base(uint32_t base, int l) {
    const int r = 8 * (l >> 4) + ((l >> 2) & 3), q = l & 3;
    return {base + off(r, q >> 1) + 8 * (q & 1), base + off(r + 4, q >> 1) + 8 * (q & 1)};
  }
  __device__ static __forceinline__ bf16x8 col(const Col &x, int kb, int c) {
    return wy::cat(wy::ld_tr((x.a ^ (32 * c)) + 32 * RB * kb), wy::ld_tr((x.b ^ (32 * c)) + 32 * RB * kb));
  }
};

// 32-index operand fragment whose rows are the matrix's columns: 16 columns
// c0 .. of an LDS matrix with `stride` bytes per row, contraction index = its
// rows r0 + 8 g .. r0 + 8 g + 7 (lane group g)
__device__ __forceinline__ bf16x8 frag_tr(uint32_t base, int stride, int r0, int c0, int l) {
  const int g = l >> 4, e = (l >> 2) & 3, q = l & 3;
  const uint32_t a = base + (r0 + 8 * g + e) * stride + 2 * (c0 + 4 * q);
  return wy::cat(wy::ld_tr(a), wy::ld_tr(a + 4 * stride));
}

// Global accesses of a workgroup go to a uniform base (scalar registers) plus a
// 32-bit byte offset per lane: the byte span of a chunk's rows, or of a state,
// stays below 2^31.
template <typename T>
__device__ __forceinline__ T ldg(const void *base, uint32_t off) {
  return *reinterpret_cast<const T *>(static_cast<const char *>(base) + off);
}
template <typename T>
__device__ __forceinline__ void stg(void *base, uint32_t off, const T &x) {
  *reinterpret_cast<T *>(static_cast<char *>(base) + off) = x;
}

// A ROWS x COLS bf16 tile staged through registers: each of the workgroup's
// THR threads holds its share as 16-byte units, zero from row L on.
template <int ROWS, int COLS, int THR>
struct Stage {
  static constexpr int UPR = COLS / 8, NU = ROWS * UPR / THR, RSTEP = THR / UPR;
  static_assert(ROWS * UPR % THR == 0 && THR % UPR == 0, "whole units and rows per thread");
  u32x4 u[NU];
  // rows of `pitch` bytes; base points at the tile's first element
  __device__ __forceinline__ void load(const bf16 *base, uint32_t pitch, int L) {
    const int r0 = threadIdx.x / UPR, c = threadIdx.x % UPR;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int r = r0 + RSTEP * i;
      u[i] = r < L ? ldg<u32x4>(base, r * pitch + 16 * c) : (u32x4)0u;
    }
  }
  // the same, but rows from L on repeat row L - 1: for tiles whose coefficients
  // are zero there
  __device__ __forceinline__ void load_clamped(const bf16 *base, uint32_t pitch, int L, uint32_t tid) {
    const uint32_t first = (tid / UPR) * pitch, last = (L - 1) * pitch, c = 16 * (tid % UPR);
#pragma unroll
    for (int i = 0; i < NU; ++i) u[i] = ldg<u32x4>(base, min(first + i * (RSTEP * pitch), last) + c);
  }
  // into columns c0 .. of a swizzled matrix of WIDTH columns
  template <int WIDTH>
  __device__ __forceinline__ void store_swz(uint32_t lds, uint32_t tid, int c0 = 0) const {
    const int r0 = tid / UPR, c = tid % UPR;
#pragma unroll
    for (int i = 0; i < NU; ++i) wy::st(lds + Swz<WIDTH>::off(r0 + RSTEP * i, c0 / 8 + c), u[i]);
  }
  template <int STRIDE>
  __device__ __forceinline__ void store(bf16 *lds) const {
    const int r0 = threadIdx.x / UPR, c = threadIdx.x % UPR;
#pragma unroll
    for (int i = 0; i < NU; ++i) *reinterpret_cast<u32x4 *>(lds + (r0 + RSTEP * i) * STRIDE + 8 * c) = u[i];
  }
};

// row-major fragment: 8 elements of row r from column c on
__device__ __forceinline__ bf16x8 frag_row(const bf16 *lds, int stride, int r, int c) {
  return *reinterpret_cast<const bf16x8 *>(lds + r * stride + c);
}

}  // namespace dn
