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

// The scales and biases of four consecutive channels; those past n repeat the
// last one and are never stored.
struct Channels {
  float scale[4], bias[4];
};

__device__ __forceinline__ Channels load_channels(const GemmArgs &g, int n0) {
  Channels c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + i, g.n - 1);
    c.scale[i] = g.w_scale[n];
    c.bias[i] = g.bias ? g.bias[n] : 0.0f;
  }
  return c;
}

// Outputs n0 .. n0 + 3 of row m, from their int32 sums.
__device__ __forceinline__ void put4(uint16_t *p, const uint16_t (&v)[4]) {
  *reinterpret_cast<words2 *>(p) = words2{(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16};
}
__device__ __forceinline__ void put4(float *p, const float (&v)[4]) {
  *reinterpret_cast<floats4 *>(p) = floats4{v[0], v[1], v[2], v[3]};
}

template <typename E>
__device__ __forceinline__ void store_outputs(const GemmArgs &g, int m, int n0, float a_scale, const Channels &c, i32x4 acc) {
  typedef typename E::raw raw;
  if (m >= g.m) return;
  raw out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = E::round((float)acc[i] * a_scale * c.scale[i] + c.bias[i]);
  raw *p = (raw *)g.y + (int64_t)m * g.ldy + n0;
  if (n0 + 4 <= g.n) {
    put4(p, out);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < g.n) p[i] = out[i];
  }
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
    const int m = m0 + 16 * t + r;
    store_outputs<E>(g, m, n0 + 4 * c, g.a_scale[min(m, g.m - 1)], load_channels(g, n0 + 4 * c), s);
  }
}

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

#define FB_LDS __attribute__((address_space(3)))
#define FB_GLB __attribute__((address_space(1)))

// Sixteen bytes per lane from global memory straight into LDS: lane l's piece, at
// base + soff + voff, lands at dst + 16 l.  A buffer load rather than a global
// one: the compiler takes a direct global load for an LDS access too and would
// then wait for all fragment reads in flight wherever it waits for some.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t *base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, 0xffffffff, 0x00027000);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t base, uint32_t voff, uint32_t soff, FB_LDS int8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (FB_LDS void *)dst, 16, voff, soff, 0, 0);
}

// LDS-tiled product: BN channels x BM tokens per workgroup, WN x WM waves, 128
// bytes of k per stage, two stages in LDS.  A stage keeps each row's eight
// 16-byte pieces at positions exchanged by the row's number (piece p of row r
// at p ^ (r % 8)), so that the lanes of a fragment read, which take one piece
// of consecutive rows, spread over the banks; the exchange is made in the
// global addresses, since a direct load writes LDS in lane order.
template <typename E, int BN, int BM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void gemm_w8a8_tile_kernel(const GemmArgs g) {
  constexpr int KB = 128, W = WN * WM, STEPS = KB / 32;
  constexpr int NT = BN / WN / 32, MT = BM / WM / 32;  // 32 x 32 tiles of a wave
  constexpr int LW = BN / 8 / W, LA = BM / 8 / W;      // direct loads (8 rows each) of a wave per stage
  static_assert(BN % (8 * W) == 0 && BM % (8 * W) == 0, "rows divide over the waves");
  // two arrays, so that the compiler sees that reads of one stage do not wait
  // for the direct loads of the other
  __shared__ __align__(1024) int8_t buf0[(BN + BM) * KB];
  __shared__ __align__(1024) int8_t buf1[(BN + BM) * KB];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // Workgroups go to the 8 XCDs in turn: each XCD takes a contiguous eighth of
  // the tiles, in panels of kPanel token blocks, so that the workgroups that
  // share an L2 share operands.
  constexpr int kPanel = 4;
  const int nb = (g.n + BN - 1) / BN, mb = (g.m + BM - 1) / BM;
  int t0;
  {
    const int total = nb * mb, xcd = blockIdx.x % 8, pos = blockIdx.x / 8;
    const int per = total / 8, rest = total % 8;
    t0 = xcd * per + min(xcd, rest) + pos;
  }
  const int panel = t0 / (kPanel * nb), in = t0 % (kPanel * nb), wide = min(kPanel, mb - panel * kPanel);
  const int n0 = in / wide * BN, m0 = (panel * kPanel + in % wide) * BM;
  const int last = (g.k - 1) / 16 * 16;
  const int piece = ((lane % 8) ^ (lane / 8)) * 16;
  // a uniform base and a 32-bit offset per lane (the host keeps 256 strides
  // below 2^31); rows past the matrix repeat its last one
  const __amdgpu_buffer_rsrc_t from_w = buffer_of(g.w + n0 * g.ldw), from_a = buffer_of(g.a + m0 * g.lda);
  uint32_t off_w[LW], off_a[LA];
#pragma unroll
  for (int i = 0; i < LW; ++i) off_w[i] = (uint32_t)min((wave * LW + i) * 8 + lane / 8, g.n - 1 - n0) * (uint32_t)g.ldw;
#pragma unroll
  for (int i = 0; i < LA; ++i) off_a[i] = (uint32_t)min((wave * LA + i) * 8 + lane / 8, g.m - 1 - m0) * (uint32_t)g.lda;
  auto fetch = [&](int stage, int8_t *buf) {
    const int k0 = stage * KB;
    const uint32_t at = min(piece, last - k0);
    FB_LDS int8_t *dst = (FB_LDS int8_t *)buf;
#pragma unroll
    for (int i = 0; i < LW; ++i) load_to_lds(from_w, off_w[i] + at, k0, dst + (wave * LW + i) * 1024);
#pragma unroll
    for (int i = 0; i < LA; ++i) load_to_lds(from_a, off_a[i] + at, k0, dst + BN * KB + (wave * LA + i) * 1024);
  };
  const int stages = (g.k + KB - 1) / KB;
  // Where k ends inside a stage, the tokens' pieces behind it are cleared (what
  // the weights hold there is multiplied with these zeros).
  auto clear_tail = [&](int8_t *buf) {
    const int left = g.k - (stages - 1) * KB;
    for (int i = threadIdx.x; i < BM * 8; i += 64 * W) {
      const int row = BN + i / 8, p = i % 8;
      i32x4 *at = reinterpret_cast<i32x4 *>(buf + row * KB + ((p ^ (row % 8)) * 16));
      if (p * 16 + 16 > left) *at = mask_tail(*at, p * 16, left);
    }
  };
  const int wn = wave / WM, wm = wave % WM;
  const int r = lane % 32, half = lane / 32;
  i32x16 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x16{};
  i32x4 wv[2][NT], av[2][MT];
  auto load_step = [&](const int8_t *buf, int s, int set) {
    const int p = 2 * s + half;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int row = (wn * NT + i) * 32 + r;
      wv[set][i] = *reinterpret_cast<const i32x4 *>(buf + row * KB + ((p ^ (row % 8)) * 16));
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int row = BN + (wm * MT + j) * 32 + r;
      av[set][j] = *reinterpret_cast<const i32x4 *>(buf + row * KB + ((p ^ (row % 8)) * 16));
    }
  };
  auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[set][i], av[set][j], acc[i][j], 0, 0, 0);
  };
  // One stage: its fragments are read one step ahead of the products, all reads
  // of a step before its products, so that they land while the products run.
  // The barrier that ends the stage's reads and the next stage's loads stands
  // before the last step's products, which cover the first reads after it.
  auto run_stage = [&](int t, int8_t *cur, int8_t *nxt, auto more) {
    if (more()) fetch(t + 1, nxt);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s + 1 < STEPS; ++s) {
      load_step(cur, s + 1, (s + 1) % 2);
      multiply(s % 2);
      __builtin_amdgcn_sched_group_barrier(0x100, NT + MT, 0);  // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x008, NT * MT, 0);  // products
      __builtin_amdgcn_sched_barrier(0);
    }
    if (more()) {
      __syncthreads();
      if (t + 2 == stages && g.k % KB) {
        clear_tail(nxt);
        __syncthreads();
      }
      load_step(nxt, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply((STEPS - 1) % 2);
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto yes = [] { return true; };
  const auto no = [] { return false; };
  fetch(0, buf0);
  __syncthreads();
  if (stages == 1 && g.k % KB) {
    clear_tail(buf0);
    __syncthreads();
  }
  load_step(buf0, 0, 0);
  int t = 0;
  for (; t + 2 < stages; t += 2) {
    run_stage(t, buf0, buf1, yes);
    run_stage(t + 1, buf1, buf0, yes);
  }
  int8_t *final = buf0;
  if (t + 1 < stages) {
    run_stage(t, buf0, buf1, yes);
    final = buf1;
  }
  run_stage(stages - 1, final, nullptr, no);
  // The epilogue's addresses are not to be computed before the loop and held in
  // registers through it.
  int ne = n0 + wn * NT * 32 + 4 * half, me = m0 + wm * MT * 32 + r;
  asm volatile("" : "+v"(ne), "+v"(me));
  // lane l of a result tile holds token l % 32, channels 8 q + 4 (l / 32) .. + 3
  float sa[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) sa[j] = g.a_scale[min(me + j * 32, g.m - 1)];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = ne + i * 32 + 8 * q;
      const Channels c = load_channels(g, n);
#pragma unroll
      for (int j = 0; j < MT; ++j)
        store_outputs<E>(g, me + j * 32, n, sa[j], c,
                         i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
      __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace fluxbin
