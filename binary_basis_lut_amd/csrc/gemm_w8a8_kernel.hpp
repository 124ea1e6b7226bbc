// gemm_w8a8_kernel.hpp -- the int8 matrix product with a scale per token and per
// output channel:
//     y[m][n] = (a_scale[m] * w_scale[n]) * sum_k a[m][k] w[n][k] + bias[n].
// The sum is exact in int32 (k <= 131071, so that even -128 * -128 products
// stay below 2^31) and therefore the same under any split of k.
#pragma once

#include "elements.hpp"

namespace fluxbin {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct GemmArgs {
  const int8_t *a, *w;
  const float *a_scale, *w_scale, *bias;  // bias may be null
  void *y;
  int64_t lda, ldw, ldy;
  int32_t m, n, k;
};

// Four consecutive outputs n0 .. n0 + 3 of row m, from their int32 sums.
template <typename E>
__device__ __forceinline__ void store_outputs(const GemmArgs &g, int m, int n0, i32x4 acc) {
  typedef typename E::raw raw;
  if (m >= g.m || n0 >= g.n) return;
  const float sa = g.a_scale[m];
  raw out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, g.n - 1);
    float v = (float)acc[i] * sa * g.w_scale[n];
    if (g.bias) v += g.bias[n];
    out[i] = E::round(v);
  }
  raw *p = (raw *)g.y + (int64_t)m * g.ldy + n0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < g.n) p[i] = out[i];
}

// The bytes [at, at + 16) of a row's k, with zeros from k on.
__device__ __forceinline__ i32x4 mask_tail(i32x4 v, int at, int k) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = k - (at + 4 * i);
    const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1;
    v[i] = (int)((uint32_t)v[i] & keep);
  }
  return v;
}

// One workgroup: 16 output channels x 16 MT tokens; its KW waves take blocks of
// 256 columns in turn and add their sums in LDS.  Both operands go from global
// memory into the registers of v_mfma_i32_16x16x64_i8: lane l holds row l % 16
// and, of each block, the 64 bytes from (l / 16) * 64 on (any order of k serves
// as long as both operands share it).
template <typename E, int MT, int KW>
__global__ __launch_bounds__(64 * KW) void gemm_w8a8_rows_kernel(const GemmArgs g) {
  constexpr int KB = 256;
  __shared__ i32x4 part[KW][MT][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int r = lane % 16, c = lane / 16;
  const int n0 = (int)blockIdx.x * 16, m0 = (int)blockIdx.y * 16 * MT;
  const int last = (g.k - 1) / 16 * 16;  // the last 16-byte piece that a row has
  const int8_t *wr = g.w + (int64_t)min(n0 + r, g.n - 1) * g.ldw;
  const int8_t *ar[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) ar[t] = g.a + (int64_t)min(m0 + 16 * t + r, g.m - 1) * g.lda;
  i32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  for (int kb = wave * KB; kb < g.k; kb += KW * KB) {
    i32x4 wv[4], av[MT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = kb + c * 64 + j * 16, from = min(at, last);
      wv[j] = *reinterpret_cast<const i32x4 *>(wr + from);
#pragma unroll
      for (int t = 0; t < MT; ++t) av[t][j] = *reinterpret_cast<const i32x4 *>(ar[t] + from);
    }
    if (kb + KB > g.k) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) av[t][j] = mask_tail(av[t][j], kb + c * 64 + j * 16, g.k);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[j], av[t][j], acc[t], 0, 0, 0);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  // lane l of a result tile holds channels 4 (l / 16) .. + 3 of token l % 16
  for (int t = wave; t < MT; t += KW) {
    i32x4 s = part[0][t][lane];
#pragma unroll
    for (int v = 1; v < KW; ++v) s += part[v][t][lane];
    store_outputs<E>(g, m0 + 16 * t + r, n0 + 4 * c, s);
  }
}

}  // namespace fluxbin
