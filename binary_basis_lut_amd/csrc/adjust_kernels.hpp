// adjust_kernels.hpp -- penalties of repeated tokens, biases and a grammar's mask
// on rows of logits, in one pass.
//
// Mathematics.  For token j of a row, c_j the times it was generated:
//     z = x > 0 ? x / rho : x rho           (tokens of the history)
//     z = z - phi c_j - pi [c_j > 0],  z = z + bias_j,  z = -inf where masked,
// in fp32, rounded once.
//
// A workgroup takes a slice of kAdjustSlice tokens of a row.  It counts the
// history's tokens of its slice in LDS (integers, so the order of the atomics
// does not show), puts the biases of its slice beside them, and then streams the
// slice through registers.  Biases of one token are added in list order by the
// first of them, so no floating-point sum depends on timing.
#pragma once

#include "elements.hpp"

namespace fluxbin {

struct AdjustArgs {
  const void *logits;
  void *out;
  const int32_t *history, *prompt_len, *total_len;     // may be null
  const float *repetition, *frequency, *presence;      // may be null
  const int32_t *bias_index;                           // may be null
  const float *bias_value;
  const uint32_t *mask;                                // may be null
  int64_t ld, ldo, ldh, ldb, ldm, rows;
  int32_t vocab, history_cols, biases, slices;
};

constexpr int kAdjustSlice = 4096;
constexpr uint32_t kGiven = 0x80000000u;  // the token is in the prompt; the low bits count its generations

template <typename E, bool BIAS, bool TINY>
__global__ __launch_bounds__(256) void adjust_logits_kernel(const AdjustArgs a) {
  typedef typename E::raw raw;
  __shared__ __align__(16) uint32_t counts[kAdjustSlice];
  __shared__ __align__(16) float bias[BIAS ? kAdjustSlice : 4];
  const int64_t row = blockIdx.x / a.slices;
  const int first = (int)(blockIdx.x % a.slices) * kAdjustSlice, n = min(a.vocab - first, kAdjustSlice);
  const int all = a.history_cols;
  const int total = a.history ? a.total_len ? max(0, min(a.total_len[row], all)) : all : 0;
  const int given = a.prompt_len ? max(0, min(a.prompt_len[row], all)) : 0;
  const float rho = a.repetition ? a.repetition[row] : 1.0f;
  const float phi = a.frequency ? a.frequency[row] : 0.0f, pi = a.presence ? a.presence[row] : 0.0f;

  if (total || BIAS) {
    for (int i = threadIdx.x; i < kAdjustSlice / 4; i += 256) {
      if (total) reinterpret_cast<uint4 *>(counts)[i] = uint4{0, 0, 0, 0};
      if (BIAS) reinterpret_cast<float4 *>(bias)[i] = float4{0, 0, 0, 0};
    }
    __syncthreads();
    const int32_t *h = a.history + row * a.ldh;
    for (int i = threadIdx.x; i < total; i += 256) {
      const uint32_t j = (uint32_t)h[i] - (uint32_t)first;
      if (j < (uint32_t)n) {
        if (i < given) atomicOr(&counts[j], kGiven);
        else atomicAdd(&counts[j], 1u);
      }
    }
    if (BIAS) {
      const int32_t *index = a.bias_index + row * a.ldb;
      const float *value = a.bias_value + row * a.ldb;
      for (int i = threadIdx.x; i < a.biases; i += 256) {
        const int32_t t = index[i];
        const uint32_t j = (uint32_t)t - (uint32_t)first;
        if (j >= (uint32_t)n) continue;
        bool leads = true;
        for (int e = 0; e < i; ++e) leads = leads && index[e] != t;
        if (!leads) continue;
        float sum = value[i];
        for (int e = i + 1; e < a.biases; ++e)
          if (index[e] == t) sum += value[e];
        bias[j] = sum;
      }
    }
    __syncthreads();
  }

  const raw *x = (const raw *)a.logits + row * a.ld;
  raw *y = (raw *)a.out + row * a.ldo;
  const uint32_t *mask = a.mask ? a.mask + row * a.ldm : nullptr;
  for (int at = first + (int)threadIdx.x * kUnit; at < first + n; at += 256 * kUnit) {
    typename E::unit u = load_part<E, TINY, int>(x, at, a.vocab, 0.0f);
    const uint32_t allowed = mask ? mask[at / 32] >> (at % 32) : ~0u;
    settle_part<E, TINY, int>(u, at, a.vocab, 0.0f);
    float f[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = u.get(i);
    if (total) {
      uint32_t c[kUnit], any = 0;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        c[i] = counts[at - first + i];
        any |= c[i];
      }
      if (any) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          const uint32_t made = c[i] & ~kGiven;
          if (c[i]) f[i] = f[i] > 0.0f ? f[i] / rho : f[i] * rho;
          if (made) f[i] = f[i] - phi * (float)made - pi;
        }
      }
    }
    if (BIAS) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) f[i] += bias[at - first + i];
    }
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = allowed >> i & 1 ? f[i] : -__builtin_inff();
    u.set(f);
    store_part<E, int>(y, at, a.vocab, u);
  }
}

}  // namespace fluxbin
