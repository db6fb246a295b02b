// Shared parts of the gated linear recurrence's kernels (gfx950).
//
// Every channel is a recurrence of its own.  With s = sigmoid(r + br),
// log a = -power softplus(lam) s, m = sqrt(1 - a^2) and u = sigmoid(i + bi) x:
//
//   h_t = a_t h_{t-1} + m_t u_t,   y = h
//
// and going back, with c the gradient that reaches h_t from later tokens (dhT at
// a sequence's last one):
//
//   g_t = dy_t + c,   c <- a_t g_t
//   W = log a dL/dlog a = g log a (a h_{t-1} - u a^2 / m)
//   dr = (1 - s) W,   di = g m u (1 - sigmoid(i + bi)),   dx = g m sigmoid(i + bi)
//   dbr = sum dr,     dbi = sum di,     dlam = sigmoid(lam) / softplus(lam) sum W
//
// Where a = 1 (a recurrence gate of minus infinity) m and W are 0 and the token
// leaves the state as it is.
//
// Both directions are composed of maps c -> A c + B, which are associative.  A
// workgroup takes 64 channels, two a lane, and walks through a segment of rows
// tile by tile.  In a tile a thread has a run of consecutive rows and composes
// their maps; one exchange through LDS then gives every run the state it starts
// from.  Each tensor is read once where the sequences times the channels fill
// the device; else sequences are cut into segments, whose maps are composed in
// a pass before.  Packed sequences are cut wherever they lie: the state in front
// of a sequence's first row is h0, and whatever reaches that row from the rows
// before is dropped, not multiplied by zero, so that nothing crosses sequences.
// Such a cut is marked by A's sign: a product of decays that has fallen to 0 drops
// nothing, and what is not finite reaches all of its sequence.
#pragma once

#include "dn_internal.h"
#include "dn_rows.h"
#include "dn_ssm.h"

namespace dn {

constexpr int GLR_CH = 64;      // channels of a workgroup
constexpr int GLR_LANES = 32;   // lanes of a row, two channels each
constexpr int GLR_THREADS = 512;
constexpr int GLR_WAVES = GLR_THREADS / 64;
constexpr int GLR_RUNS = GLR_THREADS / GLR_LANES;  // runs of rows side by side
constexpr int GLR_TILE = 128;   // rows of a segment's unit
constexpr int GLR_STATE = 64;   // rows between two states kept for the backward pass

struct GlrParams {
  const void *x, *r, *i, *dy;
  const float *lam, *br, *bi;  // br, bi may be null
  const float *h0, *dhT;       // may be null
  const int32_t *cu;           // packed sequences, or null: N sequences of T rows
  void *y, *dx, *dr, *di;      // y may be null
  float *hT, *dh0;             // may be null
  float *states;               // state entering each block of GLR_STATE rows (may be null forwards)
  float *sum_f, *sum_r;        // maps of the segments, [segment][A, B][C]
  float *part;                 // [segment][dlam, dbr, dbi][C]
  float *dlam, *dbr, *dbi;     // dbr, dbi may be null
  int64_t rows;
  int T, N, C, groups;         // groups: of GLR_CH channels
  int flat;                    // segments run over all rows; else they lie in one sequence, NS to each
  int NS, segt, nseg;          // segt: tiles of a segment
  int cut;                     // segments continue one another
  int zero_tail;
  float power;
};

hipError_t launch_glr_sum(const GlrParams &p, int dtype, bool backward, hipStream_t stream);
hipError_t launch_glr_fwd(const GlrParams &p, int dtype, hipStream_t stream);
hipError_t launch_glr_bwd(const GlrParams &p, int dtype, hipStream_t stream);

struct GlrStepParams {
  const void *x, *r, *i;
  const float *lam, *br, *bi;
  float *state;
  void *y;
  int B, C;
  float power;
};
hipError_t launch_glr_step(const GlrStepParams &p, int dtype, hipStream_t stream);

// ------------------------------------------------------------------ device

constexpr float GLR_LOG2E = 1.44269504088896340736f, GLR_LN2 = 0.69314718055994530942f;

template <typename E> struct Pair;  // two neighbouring channels
template <> struct Pair<bf16> { typedef bf16x2v type; };
template <> struct Pair<float> { typedef f32x2 type; };

template <typename E>
__device__ __forceinline__ f32x2 to_f2(typename Pair<E>::type v) {
  return (f32x2){to_f<E>(v[0]), to_f<E>(v[1])};
}
template <typename E>
__device__ __forceinline__ typename Pair<E>::type to_e2(f32x2 v) {
  if constexpr (std::is_same<E, bf16>::value) return __builtin_bit_cast(bf16x2v, pk_bf16(v[0], v[1]));
  else return v;
}

// What a channel's gates need: log2 of the decay at an open gate, and the biases
// in units of -log2 e.
struct GlrChannel {
  float k2, br, bi;
};
__device__ __forceinline__ GlrChannel glr_channel(const float *lam, const float *br, const float *bi, float power, int c) {
  // finite, so that a closed gate's 0 times it is 0
  const float k2 = -power * (GLR_LOG2E * softplus(lam[c]));
  return {k2 < -3.4e38f ? -3.4e38f : k2, br ? -GLR_LOG2E * br[c] : 0.f, bi ? -GLR_LOG2E * bi[c] : 0.f};
}

// sigmoid(z + bias), bias in units of -log2 e
__device__ __forceinline__ float glr_sigmoid(float z, float bias) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(__builtin_fmaf(z, -GLR_LOG2E, bias)));
}

// A choice that stays one: for a condition that differs between lanes the compiler
// would branch around the side that costs more, and wait at each.
__device__ __forceinline__ float glr_pick(bool first, float a, float b) {
  asm("" : "+v"(a), "+v"(b));
  return first ? a : b;
}

// 1 - a^2 for a = 2^l2, l2 <= 0: above l2 = -1/2, where the difference would lose
// digits, 2 a sinh(-log a), its sinh by the series' terms up to the fifth power with the
// seventh's best share added (the rest is below 2^-26 of it); the logarithm's ln 2 is in
// the numbers.
__device__ __forceinline__ float glr_rest(float a, float l2) {
  const float w = l2 * l2;
  float q = __builtin_fmaf(w, -0.00267815118f, -0.111007145f);
  q = __builtin_fmaf(w, q, -1.38629438f);
  return glr_pick(l2 > -0.5f, a * l2 * q, __builtin_fmaf(-a, a, 1.f));
}

// A map that starts anew has A = GLR_CUT, and compositions with it a negative A;
// decays are positive or 0.  (One that is not a number may have either sign: its B is not
// a number either, and so is the result.)
constexpr float GLR_CUT = -0.f;
__device__ __forceinline__ uint32_t glr_sign(float a) { return __builtin_bit_cast(uint32_t, a) & 0x80000000u; }

// A c + B, or B alone, whatever c is, behind a cut; DROP false where segments lie in one
// sequence, and there is nothing to drop.
template <bool DROP = true>
__device__ __forceinline__ f32x2 glr_map(f32x2 A, f32x2 c, f32x2 B) {
  const f32x2 r = {__builtin_fmaf(A[0], c[0], B[0]), __builtin_fmaf(A[1], c[1], B[1])};
  return DROP ? (f32x2){glr_sign(A[0]) ? B[0] : r[0], glr_sign(A[1]) ? B[1] : r[1]} : r;
}
// The A of two maps' composition: their product, with a cut that no product undoes, be it
// another cut's or NaN.
__device__ __forceinline__ float glr_times(float a, float b) {
  const float r = a * b;
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r) | glr_sign(a) | glr_sign(b));
}
template <bool DROP = true>
__device__ __forceinline__ f32x2 glr_times(f32x2 a, f32x2 b) {
  if (!DROP) return (f32x2){a[0] * b[0], a[1] * b[1]};
  return (f32x2){glr_times(a[0], b[0]), glr_times(a[1], b[1])};
}
__device__ __forceinline__ f32x2 glr_fma(f32x2 a, f32x2 b, f32x2 c) {
  return (f32x2){__builtin_fmaf(a[0], b[0], c[0]), __builtin_fmaf(a[1], b[1], c[1])};
}

// The sequence of a row: number n, rows [beg, end).  Behind the last packed
// sequence n = N and there is no end.
struct GlrSeq {
  int n;
  int64_t beg, end;
  // for a row that all lanes of the wave share, and all of them active: every lane looks
  // at one offset a step (up to 63 sequences one step, to 4095 two; a search by halves waits
  // for each of its loads: 1357 rows of 60 sequences 53.5 us both ways, so 51.8, 8192 of 300
  // 86 and 83)
  __device__ __forceinline__ void find(const GlrParams &p, int64_t row) {
    if (p.cu) {
      uint32_t lo = 0, hi = (uint32_t)p.N + 1;  // the first offset behind the row is one of [lo, hi]
      while (lo < hi) {
        const uint32_t step = (hi - lo + 63) / 64, at = lo + (lane_id() + 1) * step - 1;
        const uint64_t behind = __ballot(at >= hi || p.cu[at] > row);
        const uint32_t k = behind ? __builtin_ctzll(behind) : 64;
        hi = min(hi, lo + (k + 1) * step - 1);
        lo = min(hi, lo + k * step);
      }
      n = lo < 1 ? 0 : (int)lo - 1;
      beg = p.cu[n];
      end = n < p.N ? p.cu[n + 1] : INT64_MAX;
    } else {
      n = (int)(row / p.T);
      beg = (int64_t)n * p.T;
      end = beg + p.T;
    }
  }
  // on to the sequence of a later row
  __device__ __forceinline__ void walk(const GlrParams &p, int64_t row) {
    while (row >= end) {
      ++n;
      beg = end;
      end = n >= p.N ? INT64_MAX : p.cu ? p.cu[n + 1] : beg + p.T;
    }
  }
  // back to the sequence of an earlier row
  __device__ __forceinline__ void back(const GlrParams &p, int64_t row) {
    while (row < beg && n > 0) {
      --n;
      end = beg;
      beg = p.cu ? p.cu[n] : end - p.T;
    }
  }
};

// A segment's rows [row0, row1) and the number of its first block of states.
struct GlrSegment {
  int64_t row0, row1, state0;
};
__device__ __forceinline__ GlrSegment glr_segment(const GlrParams &p, int seg) {
  GlrSegment s;
  const int64_t span = (int64_t)p.segt * GLR_TILE;
  if (p.flat) {
    s.row0 = seg * span;
    s.row1 = min(s.row0 + span, p.rows);
    s.state0 = s.row0 / GLR_STATE;
  } else {
    const int n = seg / p.NS, k = seg - n * p.NS;
    s.row0 = (int64_t)n * p.T + k * span;
    s.row1 = min(s.row0 + span, (int64_t)(n + 1) * p.T);
    s.state0 = (int64_t)n * ((p.T + GLR_STATE - 1) / GLR_STATE) + k * (span / GLR_STATE);
  }
  return s;
}
// The sequence of its first row (BACK: its last one), and that sequence's first (last) segment.
template <bool BACK>
__device__ __forceinline__ int glr_reach(const GlrParams &p, const GlrSegment &s, int seg, GlrSeq &q) {
  if (!p.flat) {
    q.n = seg / p.NS;
    q.beg = (int64_t)q.n * p.T;
    q.end = q.beg + p.T;
    return BACK ? q.n * p.NS + p.NS - 1 : q.n * p.NS;
  }
  q = {};
  if (s.row0 >= s.row1) return seg;
  q.find(p, BACK ? s.row1 - 1 : s.row0);
  if (!p.cut || q.n >= p.N) return seg;
  const int64_t span = (int64_t)p.segt * GLR_TILE;
  return BACK ? (int)min((int64_t)p.nseg - 1, (q.end - 1) / span) : (int)max((int64_t)0, q.beg / span);
}

// The rows of a run that need care: bit j of `starts` (`ends`) where row j is its
// sequence's first (last), of `dead` where it lies behind the last sequence or
// behind the segment's end (`live` rows are left of the latter).
struct GlrFlags {
  uint32_t starts, ends, dead;
  int live;
};
template <int ROWS>
__device__ __forceinline__ bool glr_flags(const GlrParams &p, GlrSeq &q, int64_t row, int64_t row1, GlrFlags &f) {
  f.starts = f.ends = f.dead = 0;
  f.live = ROWS;
  q.walk(p, row);
  if (row > q.beg && row + ROWS < q.end && row + ROWS <= row1 && q.n < p.N) return false;
  const int64_t left = row1 - row;
  f.live = left < 0 ? 0 : left < ROWS ? (int)left : ROWS;
  GlrSeq w = q;
  for (int j = 0; j < f.live; ++j) {
    w.walk(p, row + j);
    if (w.n >= p.N) f.dead |= 1u << j;
    else {
      if (row + j == w.beg) f.starts |= 1u << j;
      if (row + j == w.end - 1) f.ends |= 1u << j;
    }
  }
  return true;
}

// A pointer that all lanes share, as the scalar base of an access with a 32-bit offset.
#define GLR_GLOBAL __attribute__((address_space(1)))
__device__ __forceinline__ GLR_GLOBAL char *glr_base(const void *src, int64_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(src) + bytes;
  uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  uint64_t r = (uint64_t)hi << 32 | lo;
  asm("" : "+s"(r));
  return reinterpret_cast<GLR_GLOBAL char *>(r);
}

// Byte offsets of a run's ROWS rows from a tile's first, of which `left` are there;
// those behind repeat the last one (an offset is the larger the later the row).
// Opaque, as the compiler would widen them to 64 bits far from the accesses.
template <int ROWS>
__device__ __forceinline__ void glr_offsets(uint32_t (&o)[ROWS], int at, int left, uint32_t pitch, uint32_t col) {
  const uint32_t last = (left - 1) * pitch + col;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    o[j] = min((at + j) * pitch + col, last);
    asm volatile("" : "+v"(o[j]));
  }
}

// The rows of a run, two channels a lane, from a tile's first row on that all lanes share.
template <typename E, int ROWS>
__device__ __forceinline__ void glr_load(const void *src, int64_t tile, const uint32_t (&o)[ROWS], int C,
                                         typename Pair<E>::type (&v)[ROWS]) {
  GLR_GLOBAL char *base = glr_base(src, tile * C * (int)sizeof(E));
#pragma unroll
  for (int j = 0; j < ROWS; ++j) v[j] = *reinterpret_cast<GLR_GLOBAL const typename Pair<E>::type *>(base + o[j]);
}
// The same where lanes differ in the rows: row j of `left` from `row` on.
template <typename E, int ROWS>
__device__ __forceinline__ void glr_load_at(const void *src, int64_t row, int left, int C, int c,
                                            typename Pair<E>::type (&v)[ROWS]) {
  const E *base = static_cast<const E *>(src) + row * C + c;
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
    v[j] = *reinterpret_cast<const typename Pair<E>::type *>(base + (int64_t)min(j, left - 1) * C);
}

// Stores of results, past the caches, where the inputs' maps were read and they are read
// again (whole calls, forwards + backwards: 16384 rows of 2048 channels in bf16, backwards
// alone, 131 us, with ordinary stores 140; 4 x 4096 rows of 4096 channels 125 + 210 and
// 126 + 214).
template <typename P2>
__device__ __forceinline__ void glr_store(GLR_GLOBAL char *base, uint32_t at, P2 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<GLR_GLOBAL P2 *>(base + at));
}

// All of the wave's loads and stores done.  The compiler counts the operations behind
// a load to wait for it alone, and where ways meet it takes the fewest: the walks'
// first tiles and careful rows end with this, so that the usual rows' loads do not
// wait for the stores behind them.
__device__ __forceinline__ void glr_settle() { __builtin_amdgcn_s_waitcnt(0x0f70); }

__device__ __forceinline__ f32x2 other_half(f32x2 v) {
  return (f32x2){__shfl_xor(v[0], 32, 64), __shfl_xor(v[1], 32, 64)};
}

// Composes the maps of the segments [from, to), in order or (BACK) from the last
// to the first, and applies them to zero: the waves take contiguous parts.
template <bool BACK>
__device__ __forceinline__ f32x2 glr_join(const GlrParams &p, const float *sums, int from, int to, int c, f32x4 *lds) {
  const int lane = threadIdx.x % GLR_LANES, wave = wave_id();
  const int per = (to - from + GLR_WAVES - 1) / GLR_WAVES;
  const int lo = min(from + wave * per, to), hi = min(lo + per, to);
  f32x2 A = {1.f, 1.f}, B = {0.f, 0.f};
  for (int k = 0; k < hi - lo; ++k) {
    const float *m = sums + (size_t)(BACK ? hi - 1 - k : lo + k) * 2 * p.C + c;
    const f32x2 a = *reinterpret_cast<const f32x2 *>(m), b = *reinterpret_cast<const f32x2 *>(m + p.C);
    A = glr_times(a, A);
    B = glr_map(a, B, b);
  }
  if ((threadIdx.x & 32) == 0) lds[wave * GLR_LANES + lane] = (f32x4){A[0], A[1], B[0], B[1]};
  __syncthreads();
  f32x2 r = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < GLR_WAVES; ++k) {
    const f32x4 m = lds[(BACK ? GLR_WAVES - 1 - k : k) * GLR_LANES + lane];
    r = glr_map((f32x2){m[0], m[1]}, r, (f32x2){m[2], m[3]});
  }
  __syncthreads();
  return r;
}

}  // namespace dn
