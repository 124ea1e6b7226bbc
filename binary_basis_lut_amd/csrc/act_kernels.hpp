// act_kernels.hpp -- activations to 8 bits: row quantisation, and the residual
// addition with the root-mean-square norm whose result is kept in the
// activation type, in int8, or both.
//
// Mathematics.  For a row h (for the norm: h = the residual sum as the stream
// holds it, rounded to the activation type) and weights w,
//     y_j = h_j w_j / sqrt(mean(h^2) + eps)
//     a   = max_j |t_j|,  t_j = h_j w_j   (row quantisation: t_j = x_j)
//     q_j = rint(t_j * (127 / a)),  scale = (a / 127) / sqrt(mean(h^2) + eps).
// The root is a common factor of the row, so it cancels in q: the integers
// follow from t and its largest magnitude alone, both exact under any order of
// reduction, and the sum of squares (fp32, in a fixed order) enters the scale
// only.  Both reductions need the row once, so a row is read once, held in
// registers and reduced behind one barrier.
#pragma once

#include "elements.hpp"
#include "wave_ops.hpp"

namespace fluxbin {

struct ActArgs {
  const void *x, *residual, *weight;  // residual, weight may be null (weight null: row quantisation)
  void *residual_out, *y;             // may be null
  int8_t *q;                          // may be null
  float *scale;
  int64_t ldx, ldr, ldro, ldy, ldq;
  int64_t rows, cols;
  float eps, inv_cols;
};

// The largest magnitude of a row counts as at least 2^-100, so that 127 / a
// stays finite; only bf16 and fp32 rows can be that small, and an all-zero row
// gets q = 0.
constexpr float kAmaxFloor = 7.888609052210118e-31f;

struct RowScale {
  float inv;   // 1 / sqrt(mean(h^2) + eps), NaN if that sum is not finite; 1 without a norm
  float mul;   // 127 / a
  float scale; // NaN if the row holds a value whose t is not finite
  bool finite;
};

// abits: the bits of the largest |t| as an unsigned integer, whose order is
// that of the magnitudes with NaN above infinity.
__device__ __forceinline__ RowScale row_scale(float ss, uint32_t abits, bool norm, float inv_cols, float eps) {
  RowScale r;
  r.finite = abits < 0x7f800000u;
  const float a = fmaxf(__builtin_bit_cast(float, abits), kAmaxFloor);
  r.inv = 1.0f;
  if (norm) r.inv = ss < __builtin_inff() ? 1.0f / sqrtf(fmaf(ss, inv_cols, eps)) : __builtin_nanf("");
  r.mul = 127.0f / a;
  r.scale = r.finite ? (a / 127.0f) * r.inv : __builtin_nanf("");
  return r;
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7fffffffu; }

template <typename I>
__device__ __forceinline__ void store_q(int8_t *row, I at, I n, const float (&t)[kUnit], const RowScale &r) {
  uint32_t b[kUnit];
#pragma unroll
  for (int i = 0; i < kUnit; ++i) b[i] = r.finite ? (uint32_t)(int)rintf(t[i] * r.mul) & 0xffu : 0u;
  if (at + kUnit <= n) {
    bytes8 w;
    w.x = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    w.y = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
    *reinterpret_cast<bytes8 *>(row + at) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if (at + i < n) row[at + i] = (int8_t)b[i];
  }
}

// A thread's unit of a row: adds the residual, keeps the sum as h, and joins the
// sum of squares and the largest |t|.
template <typename E, bool NORM>
__device__ __forceinline__ void take_unit(typename E::unit &h, const typename E::unit &res, const typename E::unit &w, bool add,
                                          float &ss, uint32_t &ab) {
  if (NORM && add) {
    float f[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = h.get(i) + res.get(i);
    h.set(f);
  }
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    const float v = h.get(i);
    if (NORM) ss = fmaf(v, v, ss);
    ab = max(ab, abs_bits(NORM ? v * w.get(i) : v));
  }
}

// Writes a unit's y and q.
template <typename E, bool NORM, typename I>
__device__ __forceinline__ void give_unit(const ActArgs &a, int64_t row, I at, const typename E::unit &h,
                                          const typename E::unit &w, const RowScale &rs) {
  typedef typename E::raw raw;
  float t[kUnit];
#pragma unroll
  for (int i = 0; i < kUnit; ++i) t[i] = NORM ? h.get(i) * w.get(i) : h.get(i);
  if (a.q) store_q<I>(a.q + row * a.ldq, at, (I)a.cols, t, rs);
  if (NORM && a.y) {
    typename E::unit y;
    float f[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = h.get(i) * rs.inv * w.get(i);
    y.set(f);
    store_part<E, I>((raw *)a.y + row * a.ldy, at, (I)a.cols, y);
  }
}

// Memory-bound: a row is read once and its results written once, and what
// matters is how many bytes of how many rows a CU has in flight, so the row's
// units stay in registers as they are stored.  MI355X: 8192 x 8192 fp16 with a
// residual (470 MB) 81 - 87 us = 5.4 - 5.8 TB/s, kept in fp16 instead of int8
// (537 MB) 95 us, 4096 x 4096 24.4 us; fp16 to int8 alone, 8192 x 28672 (705 MB)
// 130 - 144 us = 4.9 - 5.4 TB/s, 30000 x 4000 66 us; one row of 4096 3.5 us against
// 1.6 us of an empty launch.  The norm of up to 8192 columns takes up to 77
// registers (fp32 103); of more columns its three tensors' units are more than
// the registers hold (12 spilled at 1024 x 2 in 16 bits, held to eight waves per
// SIMD; 22 - 36 at 1024 x 4), and it is slower: 4000 x 11008 fp16 81 us =
// 3.8 TB/s, 2000 x 16384 54 us = 4.3, 1000 x 28672 70 us = 2.9 TB/s.
//
// TPR threads per row (64: one wave, several rows to a workgroup), U units of
// eight elements per thread; the row has at least 8 and at most TPR * U * 8
// columns.
template <typename E, bool NORM, int TPR, int U>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR)
__attribute__((amdgpu_waves_per_eu(TPR == 1024 && U <= 2 && sizeof(typename E::raw) == 2 ? 8 : 1))) void act_rows_kernel(const ActArgs a) {
  typedef typename E::raw raw;
  constexpr int TPB = TPR < 256 ? 256 : TPR, RPB = TPB / TPR, WPR = TPR / 64;
  __shared__ float s_ss[TPB / 64];
  __shared__ uint32_t s_ab[TPB / 64];
  const int lane = threadIdx.x % TPR, slot = RPB == 1 ? 0 : threadIdx.x / TPR;
  const bool add = NORM && a.residual;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + slot;
    const bool live = row < a.rows;
    const int n = live ? (int)a.cols : 0;
    const raw *x = (const raw *)a.x + row * a.ldx, *res = (const raw *)a.residual + row * a.ldr;
    const raw *wt = (const raw *)a.weight;
    typename E::unit h[U], rv[U], wv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (u * TPR + lane) * kUnit;
      h[u] = load_part<E, false, int>(x, at, n, 0.0f);
      if (add) rv[u] = load_part<E, false, int>(res, at, n, 0.0f);
      if (NORM) wv[u] = load_part<E, false, int>(wt, at, n, 0.0f);
    }
    float ss = 0.0f;
    uint32_t ab = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (u * TPR + lane) * kUnit;
      settle_part<E, false, int>(h[u], at, n, 0.0f);
      if (add) settle_part<E, false, int>(rv[u], at, n, 0.0f);
      if (NORM) settle_part<E, false, int>(wv[u], at, n, 0.0f);
      take_unit<E, NORM>(h[u], rv[u], wv[u], add, ss, ab);
      if (NORM && a.residual_out) store_part<E, int>((raw *)a.residual_out + row * a.ldro, at, n, h[u]);
      if (NORM) {
        h[u].hold();
        wv[u].hold();
      }
    }
    if (NORM) ss = wave_reduce<SumF>(ss);
    ab = wave_reduce<MaxU>(ab);
    if (WPR > 1) {
      if (threadIdx.x % 64 == 0) {
        s_ss[threadIdx.x / 64] = ss;
        s_ab[threadIdx.x / 64] = ab;
      }
      __syncthreads();
      ss = 0.0f;
      ab = 0;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        ss += s_ss[i];
        ab = max(ab, s_ab[i]);
      }
      __syncthreads();  // the next row writes the partials again
    }
    const RowScale rs = row_scale(ss, ab, NORM, a.inv_cols, a.eps);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (u * TPR + lane) * kUnit;
      if (at < n) give_unit<E, NORM, int>(a, row, at, h[u], wv[u], rs);
    }
    if (live && a.q && lane == 0) a.scale[row] = rs.scale;
  }
}

// Rows beyond the registers of a workgroup, and rows shorter than a unit: two
// passes over the row, the second one from the caches.
template <typename E, bool NORM, bool TINY>
__global__ __launch_bounds__(1024) void act_long_rows_kernel(const ActArgs a) {
  typedef typename E::raw raw;
  constexpr int W = 16;
  __shared__ float s_ss[W];
  __shared__ uint32_t s_ab[W];
  const int64_t n = a.cols;
  const raw *wt = (const raw *)a.weight;
  const bool add = NORM && a.residual;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const raw *x = (const raw *)a.x + row * a.ldx, *res = (const raw *)a.residual + row * a.ldr;
    float ss = 0.0f;
    uint32_t ab = 0;
    for (int64_t at = (int64_t)threadIdx.x * kUnit; at < n; at += 1024 * kUnit) {
      typename E::unit h = load_part<E, TINY, int64_t>(x, at, n, 0.0f), rv, wv;
      if (add) rv = load_part<E, TINY, int64_t>(res, at, n, 0.0f);
      if (NORM) wv = load_part<E, TINY, int64_t>(wt, at, n, 0.0f);
      settle_part<E, TINY, int64_t>(h, at, n, 0.0f);
      if (add) settle_part<E, TINY, int64_t>(rv, at, n, 0.0f);
      if (NORM) settle_part<E, TINY, int64_t>(wv, at, n, 0.0f);
      take_unit<E, NORM>(h, rv, wv, add, ss, ab);
    }
    if (NORM) ss = wave_reduce<SumF>(ss);
    ab = wave_reduce<MaxU>(ab);
    if (threadIdx.x % 64 == 0) {
      s_ss[threadIdx.x / 64] = ss;
      s_ab[threadIdx.x / 64] = ab;
    }
    __syncthreads();
    ss = 0.0f;
    ab = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      ss += s_ss[i];
      ab = max(ab, s_ab[i]);
    }
    __syncthreads();
    const RowScale rs = row_scale(ss, ab, NORM, a.inv_cols, a.eps);
    for (int64_t at = (int64_t)threadIdx.x * kUnit; at < n; at += 1024 * kUnit) {
      // residual_out may be x or residual itself: a thread reads its elements
      // again before it writes them (of a last unit's others it keeps none)
      typename E::unit h = load_part<E, TINY, int64_t>(x, at, n, 0.0f), rv, wv;
      if (add) rv = load_part<E, TINY, int64_t>(res, at, n, 0.0f);
      if (NORM) wv = load_part<E, TINY, int64_t>(wt, at, n, 0.0f);
      settle_part<E, TINY, int64_t>(h, at, n, 0.0f);
      if (add) settle_part<E, TINY, int64_t>(rv, at, n, 0.0f);
      if (NORM) settle_part<E, TINY, int64_t>(wv, at, n, 0.0f);
      float ss2 = 0.0f;
      uint32_t ab2 = 0;
      take_unit<E, NORM>(h, rv, wv, add, ss2, ab2);
      if (NORM && a.residual_out) store_part<E, int64_t>((raw *)a.residual_out + row * a.ldro, at, n, h);
      give_unit<E, NORM, int64_t>(a, row, at, h, wv, rs);
    }
    if (a.q && threadIdx.x == 0) a.scale[row] = rs.scale;
  }
}

}  // namespace fluxbin
