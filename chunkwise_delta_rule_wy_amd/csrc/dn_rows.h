// Row-wise streaming helpers.  The per-(token, head) kernels read a row of Dk
// elements by Dk / N lanes, 16 bytes each (N = 8 for bf16, 4 for fp32); the
// lanes of a row sit in one wave, so row sums are lane shuffles.  The norms'
// rows are wider (Row).
#pragma once

#include "dn_internal.h"

namespace dn {

constexpr int ROW_THREADS = 256;

template <typename E> struct Vec16;  // 16 bytes of a row
template <> struct Vec16<bf16> { typedef bf16x8 type; static constexpr int N = 8; };
template <> struct Vec16<float> { typedef f32x4 type; static constexpr int N = 4; };

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) x += __shfl_xor(x, m, 64);
  return x;
}

template <typename E, int DK>
struct RowMap {
  static constexpr int PER = Vec16<E>::N;          // row elements per lane
  static constexpr int LANES = DK / PER;           // lanes per row (8 .. 32)
  static constexpr int RPB = ROW_THREADS / LANES;  // rows per workgroup
  static_assert(LANES <= 64 && 64 % LANES == 0, "a row sits in one wave");
};

template <typename E>
__device__ __forceinline__ void load_row(const E *src, float (&x)[Vec16<E>::N]) {
  const typename Vec16<E>::type v = *reinterpret_cast<const typename Vec16<E>::type *>(src);
#pragma unroll
  for (int e = 0; e < Vec16<E>::N; ++e) x[e] = to_f<E>(v[e]);
}

template <typename E>
__device__ __forceinline__ void store_row(E *dst, const float (&x)[Vec16<E>::N]) {
  typename Vec16<E>::type v;
#pragma unroll
  for (int e = 0; e < Vec16<E>::N; ++e) v[e] = to_e<E>(x[e]);
  *reinterpret_cast<typename Vec16<E>::type *>(dst) = v;
}

// fp32 row slice of N elements (N / 4 16-byte accesses)
template <int N>
__device__ __forceinline__ void load_f32(const float *src, float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const f32x4 v = *reinterpret_cast<const f32x4 *>(src + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[e + i] = v[i];
  }
}
template <int N>
__device__ __forceinline__ void store_f32(float *dst, const float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) *reinterpret_cast<f32x4 *>(dst + e) = (f32x4){x[e], x[e + 1], x[e + 2], x[e + 3]};
}

// Wide rows: a row of D values (a multiple of 8) lies in the registers of LPR
// lanes, K units of 16 bytes of E per lane; values of another type T (fp32
// beside bf16) come and go by the same units.  LPR is part of a wave, or the
// whole workgroup of ROW_THREADS.
template <typename E, int LPR, int K>
struct Row {
  static constexpr int V = Vec16<E>::N, N = K * V;
  __device__ static __forceinline__ int col(int k, int lane) { return (k * LPR + lane) * V; }
  template <typename T>
  __device__ static __forceinline__ void load(const T *src, int lane, int D, float (&x)[N]) {
    constexpr int U = Vec16<T>::N;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = col(k, lane);
      if (c < D) {
#pragma unroll
        for (int u = 0; u < V; u += U) {
          const typename Vec16<T>::type v = *reinterpret_cast<const typename Vec16<T>::type *>(src + c + u);
#pragma unroll
          for (int e = 0; e < U; ++e) x[k * V + u + e] = to_f<T>(v[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[k * V + e] = 0.f;
      }
    }
  }
  __device__ static __forceinline__ void load_w(const float *src, int lane, int D, float (&x)[N]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = col(k, lane);
#pragma unroll
      for (int e = 0; e < V; ++e) x[k * V + e] = c < D ? src[c + e] : 0.f;
    }
  }
  // PAST: past the caches, where one instruction's units fill whole lines (medians of the
  // residual addition and norm of 16384 x 4096 bf16 values forwards: 103 us, with ordinary
  // stores 108; fp32 beside bf16, whose units come by halves, 160 and 156).
  template <bool PAST = false, typename T>
  __device__ static __forceinline__ void store(T *dst, int lane, int D, const float (&x)[N]) {
    constexpr int U = Vec16<T>::N;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = col(k, lane);
      if (c >= D) continue;
#pragma unroll
      for (int u = 0; u < V; u += U) {
        typename Vec16<T>::type v;
#pragma unroll
        for (int e = 0; e < U; ++e) v[e] = to_e<T>(x[k * V + u + e]);
        auto *to = reinterpret_cast<typename Vec16<T>::type *>(dst + c + u);
        if constexpr (PAST && U == V) __builtin_nontemporal_store(v, to);
        else *to = v;
      }
    }
  }
};

// A row's units as they lie in memory, loaded ahead of their use.
template <typename E, typename T, int LPR, int K>
struct RawRow {
  using RW = Row<E, LPR, K>;
  static constexpr int U = Vec16<T>::N, PER = RW::V / U;
  typename Vec16<T>::type v[K * PER];
  // lanes behind the row's end repeat its first unit
  __device__ __forceinline__ void load(const T *src, int lane, int D) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = RW::col(k, lane), at = c < D ? c : 0;
#pragma unroll
      for (int u = 0; u < PER; ++u) v[k * PER + u] = *reinterpret_cast<const typename Vec16<T>::type *>(src + at + u * U);
    }
  }
  __device__ __forceinline__ void get(int lane, int D, float (&x)[RW::N]) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < RW::V; ++e) x[k * RW::V + e] = RW::col(k, lane) < D ? to_f<T>(v[k * PER + e / U][e % U]) : 0.f;
  }
};

// two sums over a row's lanes at once
template <int LPR>
__device__ __forceinline__ f32x2 lanes_sum2(f32x2 x, f32x2 (*buf)[ROW_THREADS / 64], int &turn) {
  constexpr int L = LPR < 64 ? LPR : 64;
  x = (f32x2){group_sum<L>(x[0]), group_sum<L>(x[1])};
  if constexpr (LPR > 64) {
    f32x2 *b = buf[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (f32x2){0.f, 0.f};
#pragma unroll
    for (int i = 0; i < LPR / 64; ++i) x = (f32x2){x[0] + b[i][0], x[1] + b[i][1]};
  }
  return x;
}

// sum (or, with MAX, maximum) over a row's lanes; a row as wide as the workgroup
// goes through LDS (two buffers taken in turn, one barrier a sum)
template <int LPR, bool MAX = false>
__device__ __forceinline__ float lanes_sum(float x, float (*buf)[ROW_THREADS / 64], int &turn) {
  if constexpr (MAX) {
#pragma unroll
    for (int m = 1; m < (LPR < 64 ? LPR : 64); m <<= 1) x = fmaxf(x, __shfl_xor(x, m, 64));
  } else {
    x = group_sum<(LPR < 64 ? LPR : 64)>(x);
  }
  if constexpr (LPR > 64) {
    float *b = buf[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < LPR / 64; ++i) s = MAX ? fmaxf(s, b[i]) : s + b[i];
    return s;
  }
  return x;
}

// Sums over the rows of a [rows][n] fp32 matrix (n a multiple of 4), for the
// second stage of a deterministic reduction: a workgroup of 256 threads takes
// 16 columns, four lanes of 16 bytes each, and 64 interleaved groups of rows,
// whose sums meet in LDS, so that even a narrow matrix has enough loads in
// flight.  Thread t < 16 gets the sum of column 16 blockIdx.x + t.
constexpr int SUM_COLS = 16;
__device__ __forceinline__ float column_sum(const float *m, int rows, int64_t n, int64_t col0) {
  __shared__ float part[64][SUM_COLS];
  const int q = threadIdx.x & 3, g = threadIdx.x >> 2;
  const int64_t c = col0 + 4 * q;
  f32x4 a = zero4();
  if (c < n) {
    int r = g;
    for (; r + 3 * 64 < rows; r += 4 * 64) {
      f32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const f32x4 *>(m + (r + 64 * i) * n + c);
      a += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; r < rows; r += 64) a += *reinterpret_cast<const f32x4 *>(m + r * n + c);
  }
  *reinterpret_cast<f32x4 *>(&part[g][4 * q]) = a;
  for (int d = 32; d > 0; d >>= 1) {
    __syncthreads();
    if (g < d) *reinterpret_cast<f32x4 *>(&part[g][4 * q]) += *reinterpret_cast<const f32x4 *>(&part[g + d][4 * q]);
  }
  __syncthreads();
  return threadIdx.x < SUM_COLS ? part[0][threadIdx.x] : 0.f;
}

}  // namespace dn
