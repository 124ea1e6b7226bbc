// adjust_kernels.hpp -- penalties of repeated tokens, biases and a grammar's mask
// on rows of logits, in one pass.
//
// Mathematics.  For token j of a row, c_j the times it was generated:
//     z = x > 0 ? x / rho : x rho           (tokens of the history)
//     z = z - phi c_j - pi [c_j > 0],  z = z + bias_j,  z = -inf where masked,
// in fp32, rounded once.
//
// A workgroup takes a slice of a row's tokens.  It counts the
// history's tokens of its slice in LDS (integers, so the order of the atomics
// does not show), puts the biases of its slice beside them, and then streams the
// slice through registers.  Biases of one token are added in list order by one
// thread, so no floating-point sum depends on timing.
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

typedef int32_t i32s4 __attribute__((ext_vector_type(4), aligned(4)));

// A token's word: it is in the prompt, it has a bias, and how often it was generated.
constexpr uint32_t kGiven = 0x80000000u, kBiased = 0x40000000u;

// The sum of every token's biases, in list order, into bias[] of the tokens then
// marked kBiased.  A token's only entry writes it; where some token has a second
// one, the first of them goes through the list again.
template <int T>
__device__ __forceinline__ void take_biases(const AdjustArgs &a, int64_t row, int first, int n, uint32_t *counts, float *bias, int *again) {
  const int32_t *index = a.bias_index + row * a.ldb;
  const float *value = a.bias_value + row * a.ldb;
  for (int i = threadIdx.x; i < a.biases; i += T) {
    const float v = value[i];
    const uint32_t j = (uint32_t)index[i] - (uint32_t)first;
    if (j >= (uint32_t)n) continue;
    if (atomicOr(&counts[j], kBiased) & kBiased) *again = 1;
    bias[j] = v;
  }
  __syncthreads();
  if (!*again) return;
  for (int i = threadIdx.x; i < a.biases; i += T) {
    const int32_t t = index[i];
    const uint32_t j = (uint32_t)t - (uint32_t)first;
    if (j >= (uint32_t)n) continue;
    float sum = value[i];
    bool leads = true;
    for (int e = 0; e < a.biases; ++e) {
      const bool same = index[e] == t;
      leads = leads && !(same && e < i);
      if (same && e > i) sum += value[e];
    }
    if (leads) bias[j] = sum;
  }
}

// -inf for the elements whose bit is 0.
template <typename E>
__device__ __forceinline__ void forbid(HalfUnit<E> &u, uint32_t bits) {
  constexpr uint32_t none = __is_same(E, F16) ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t keep = ((bits >> (2 * i) & 1) ? 0xffffu : 0u) | ((bits >> (2 * i + 1) & 1) ? 0xffff0000u : 0u);
    u.w[i] = (u.w[i] & keep) | (none & ~keep);
  }
}
template <typename E>
__device__ __forceinline__ void forbid(FloatUnit &u, uint32_t bits) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i) u.f[i] = bits >> i & 1 ? u.f[i] : -__builtin_inff();
}

// T threads, SLICE tokens.  A slice goes through the whole history, so slices are as
// large as the LDS lets two workgroups of 1024 threads be on a CU: 16384 tokens'
// words, or 8192 with their biases.  Against 256 threads and 4096 tokens
// throughout, 64 x 131072 bf16 with 4000 tokens of history and 50 biases takes
// 12.9 us for 15.4, 2048 x 32000 fp32 84 for 99 and one row of 32000 4.7 for 5.8, each
// on the same operands again; on others 16, 100 to 106 (5.1 to 5.3 TB/s) and 4.3.
template <typename E, bool BIAS, bool TINY, int T, int SLICE>
__global__ __launch_bounds__(T) void adjust_logits_kernel(const AdjustArgs a) {
  typedef typename E::raw raw;
  constexpr int kMine = SLICE / T / kUnit, kLoads = 1024 / T;
  __shared__ __align__(16) uint32_t counts[SLICE];
  __shared__ float bias[BIAS ? SLICE : 1];
  __shared__ int again;
  const int64_t row = blockIdx.x / a.slices;
  const int first = (int)(blockIdx.x % a.slices) * SLICE, n = min(a.vocab - first, SLICE);
  // The slice and its mask are asked for before the history is gone through.
  const raw *x = (const raw *)a.logits + row * a.ld;
  raw *y = (raw *)a.out + row * a.ldo;
  const uint32_t *mask = a.mask ? a.mask + row * a.ldm : nullptr;
  typename E::unit unit[kMine];
  uint32_t allowed[kMine];
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int at = first + (u * T + (int)threadIdx.x) * kUnit;
    unit[u] = load_part<E, TINY, int>(x, at, a.vocab, 0.0f);
    allowed[u] = mask && at < a.vocab ? mask[at / 32] : ~0u;
  }
  const int all = a.history_cols;
  const int total = a.history ? a.total_len ? max(0, min(a.total_len[row], all)) : all : 0;
  const int given = a.prompt_len ? max(0, min(a.prompt_len[row], all)) : 0;
  const float rho = a.repetition ? a.repetition[row] : 1.0f;
  const float phi = a.frequency ? a.frequency[row] : 0.0f, pi = a.presence ? a.presence[row] : 0.0f;

  if (a.history || BIAS) {
    for (int i = threadIdx.x; i < (n + 3) / 4; i += T) reinterpret_cast<uint4 *>(counts)[i] = uint4{0, 0, 0, 0};
    if (BIAS && threadIdx.x == 0) again = 0;
    __syncthreads();
    // four tokens a load, up to 4096 of them in flight; the columns behind
    // total_len exist, so nothing waits for it
    const int32_t *h = a.history + row * a.ldh;
    for (int base = (int)threadIdx.x * 4; base < all; base += kLoads * 4 * T) {
      i32s4 t[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int at = base + u * 4 * T;
        t[u] = i32s4{-1, -1, -1, -1};
        if (at + 4 <= all) {
          t[u] = *reinterpret_cast<const i32s4 *>(h + at);
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (at + e < all) t[u][e] = h[at + e];
        }
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = base + u * 4 * T + e;
          const uint32_t j = (uint32_t)t[u][e] - (uint32_t)first;
          if (j < (uint32_t)n && at < total) {
            if (at < given) atomicOr(&counts[j], kGiven);
            else atomicAdd(&counts[j], 1u);
          }
        }
    }
    if (BIAS) take_biases<T>(a, row, first, n, counts, bias, &again);
    __syncthreads();
  }

#pragma unroll
  for (int v = 0; v < kMine; ++v) {
    const int at = first + (v * T + (int)threadIdx.x) * kUnit;
    if (at >= first + n) continue;
    typename E::unit u = unit[v];
    settle_part<E, TINY, int>(u, at, a.vocab, 0.0f);
    const uint32_t bits = allowed[v] >> (at % 32);
    if (a.history || BIAS) {
      uint32_t c[kUnit], any = 0;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        c[i] = counts[at - first + i];
        any |= c[i];
      }
      if (any) {  // most units have no token of the history, and stay as they are stored
        float f[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          f[i] = u.get(i);
          const uint32_t made = c[i] & ~(kGiven | kBiased);
          if (c[i] & ~kBiased) f[i] = f[i] > 0.0f ? f[i] / rho : f[i] * rho;
          if (made) f[i] = f[i] - phi * (float)made - pi;
          if (BIAS && (c[i] & kBiased)) f[i] += bias[at - first + i];
        }
        u.set(f);
      }
    }
    if (mask) forbid<E>(u, bits);
    store_part<E, int>(y, at, a.vocab, u);
  }
}

}  // namespace fluxbin
