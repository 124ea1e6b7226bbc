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
  if (n0 + 4 <= g.n) {
    const floats4 s = *reinterpret_cast<const floats4 *>(g.w_scale + (uint32_t)n0);
    const floats4 b = g.bias ? *reinterpret_cast<const floats4 *>(g.bias + (uint32_t)n0) : floats4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c.scale[i] = s[i];
      c.bias[i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t n = min(n0 + i, g.n - 1);
      c.scale[i] = g.w_scale[n];
      c.bias[i] = g.bias ? g.bias[n] : 0.0f;
    }
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

// Sixteen bytes of outputs, channels n .. of a row of `end`.
__device__ __forceinline__ void store_piece(uint16_t *row, int n, int end, i32x4 v) {
  if (n + 8 <= end) {
    *reinterpret_cast<words4 *>(row + n) = words4{(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < end) row[n + i] = (uint16_t)((uint32_t)v[i / 2] >> (16 * (i % 2)));
  }
}
__device__ __forceinline__ void store_piece(float *row, int n, int end, i32x4 v) {
  int w[4] = {v[0], v[1], v[2], v[3]};
  if (n + 4 <= end) {
    *reinterpret_cast<floats4 *>(row + n) = floats4{__builtin_bit_cast(float, w[0]), __builtin_bit_cast(float, w[1]),
                                                    __builtin_bit_cast(float, w[2]), __builtin_bit_cast(float, w[3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < end) row[n + i] = __builtin_bit_cast(float, w[i]);
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

// One workgroup: 16 output channels x 16 tokens; its KW waves take blocks of
// 256 columns in turn and add their sums in LDS.  Both operands go from global
// memory into the registers of v_mfma_i32_16x16x64_i8: lane l holds row l % 16
// and, of each 64 columns, the 16 bytes from (l / 16) * 16 on.  For one or a few
// tokens the weights' HBM read is all there is to do (one token, 8192 x 28672:
// 235 MB in 40 us = 5.9 TB/s), and eight waves a workgroup keep it going.
template <typename E, int KW>
__global__ __launch_bounds__(64 * KW) void gemm_w8a8_rows_kernel(const GemmArgs g) {
  constexpr int KB = 256;
  __shared__ i32x4 part[KW][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int r = lane % 16, c = lane / 16;
  const int n0 = (int)blockIdx.x * 16, m0 = (int)blockIdx.y * 16;
  const int last = (g.k - 1) / 16 * 16;  // the last 16-byte piece that a row has
  const int8_t *wr = g.w + (int64_t)min(n0 + r, g.n - 1) * g.ldw;
  const int8_t *ar = g.a + (int64_t)min(m0 + r, g.m - 1) * g.lda;
  i32x4 acc{0, 0, 0, 0};
  for (int kb = wave * KB; kb < g.k; kb += KW * KB) {
    i32x4 wv[4], av[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int from = min(kb + j * 64 + c * 16, last);
      wv[j] = *reinterpret_cast<const i32x4 *>(wr + from);
      av[j] = *reinterpret_cast<const i32x4 *>(ar + from);
    }
    if (kb + KB > g.k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) av[j] = mask_tail(av[j], kb + j * 64 + c * 16, g.k);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[j], av[j], acc, 0, 0, 0);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int v = 1; v < KW; ++v) acc += part[v][lane];
    // lane l holds channels 4 (l / 16) .. + 3 of token l % 16
    const int m = m0 + r;
    store_outputs<E>(g, m, n0 + 4 * c, g.a_scale[min(m, g.m - 1)], load_channels(g, n0 + 4 * c), acc);
  }
}

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

#define FB_LDS __attribute__((address_space(3)))
#define FB_GLB __attribute__((address_space(1)))

// Sixteen bytes per lane from global memory straight into LDS: lane l's piece, at
// base + soff + voff, lands at dst + 16 l.  A buffer load rather than a global
// one: the compiler takes a direct global load for an LDS access too and would
// then wait for all fragment reads in flight wherever it waits for some.
// The same address, known to be the same in every lane: a buffer descriptor in
// vector registers would be read out lane by lane around every load.
__device__ __forceinline__ const int8_t *in_scalars(const int8_t *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const int8_t *>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                                          (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
// A buffer of `bytes` 0 gives zeros and touches no memory.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t base, uint32_t voff, uint32_t soff, FB_LDS int8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (FB_LDS void *)dst, 16, voff, soff, 0, 0);
}

// Waits until at most `vm` of the wave's vector-memory operations and none of
// its LDS operations are outstanding, then for the workgroup.
template <int VM>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(VM < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | (VM >> 4) << 14);  // lgkmcnt 0, expcnt any
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// LDS-tiled product: BN channels x BM tokens per workgroup, WN x WM x WK waves
// (WK of them share a wave tile and split each stage's k), KB bytes of k per
// stage, S stages in LDS of which S - 1 are loaded ahead.  A stage keeps each
// row's 16-byte pieces at positions exchanged by the row's number, so that the
// 16 lanes of a fragment read that the LDS serves at once, which take one piece
// of consecutive rows, fall into all 64 banks: piece p of row r stands at
// p ^ (r / 2 % 8) in rows of 128 bytes and at p ^ (r % 16) in rows of 256.  The
// exchange is made in the global addresses, since a direct load writes LDS in
// lane order.
//
// What bounds it: with 256 x 256 tiles the chip's power (8192 x 28672 x 8192 in 1.57
// - 1.71 ms, 2.25 - 2.45 POP/s; the products alone, on registers, 3.4 POP/s; matrix
// pipes busy 66 % of the cycles at 1.75 GHz), with small tiles the loads that a CU
// has in flight (about 55 GB/s of operands with the weights from HBM, 70
// where the caches hold them: 333 x 4096 x 11008 in 39 and 29 us), and for few tokens the HBM
// (16 x 57344 x 8192, 470 MB, at 5.6 TB/s).
//
// Fragments are read one step ahead of the products; a step is G of the wave's
// 32-byte blocks of a stage.  Large wave tiles take G = 1 (a step's products
// outlast the reads of the next), small ones all their blocks at once, so that
// a stage waits for LDS once.
template <typename E, int BN, int BM, int WN, int WM, int WK, int KB, int S, int G>
__global__ __launch_bounds__(64 * WN * WM * WK) void gemm_w8a8_tile_kernel(const GemmArgs g) {
  constexpr int W = WN * WM * WK, BLOCKS = KB / 32 / WK, STEPS = BLOCKS / G, STAGE = (BN + BM) * KB;
  constexpr int NT = BN / WN / 32, MT = BM / WM / 32;   // 32 x 32 tiles of a wave
  constexpr int PIECES = KB / 16, RPL = 64 / PIECES;    // pieces of a row; rows of a direct load
  constexpr int LW = BN / RPL / W, LA = BM / RPL / W;   // direct loads of a wave per stage
  constexpr int PERIOD = 16 / RPL;                      // direct loads after which the exchange repeats
  static_assert(KB == 128 || KB == 256, "rows of 8 or 16 pieces");
  static_assert(BN % (RPL * W) == 0 && BM % (RPL * W) == 0, "rows divide over the waves");
  static_assert(BLOCKS % G == 0 && STEPS > 0, "blocks divide into steps");
  constexpr int sums_bytes = (WK - 1) * BN * BM * 4;    // what the waves of a tile hand to the first of them
  __shared__ __align__(1024) int8_t lds[S * STAGE];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // Workgroups go to the 8 XCDs in turn: each XCD takes a contiguous eighth of
  // the tiles, in panels of kPanel token blocks, so that the workgroups that
  // share an L2 share operands.
  constexpr int kPanel = BM >= 256 ? 4 : 8;
  const int nb = (g.n + BN - 1) / BN, mb = (g.m + BM - 1) / BM;
  int tile;
  {
    const int total = nb * mb, xcd = blockIdx.x % 8, pos = blockIdx.x / 8;
    const int per = total / 8, rest = total % 8;
    tile = xcd * per + min(xcd, rest) + pos;
  }
  const int panel = tile / (kPanel * nb), in = tile % (kPanel * nb), wide = min(kPanel, mb - panel * kPanel);
  const int n0 = in / wide * BN, m0 = (panel * kPanel + in % wide) * BM;
  const int last = (g.k - 1) / 16 * 16;
  // The loads' uniform bases and 32-bit offsets per lane (the host keeps 256
  // strides below 2^31); rows past the matrix repeat its last one.
  const int8_t *base_w = in_scalars(g.w + n0 * g.ldw), *base_a = in_scalars(g.a + m0 * g.lda);
  uint32_t off_w[LW], off_a[LA];
#pragma unroll
  for (int i = 0; i < LW; ++i) off_w[i] = (uint32_t)min((wave * LW + i) * RPL + lane / PIECES, g.n - 1 - n0) * (uint32_t)g.ldw;
#pragma unroll
  for (int i = 0; i < LA; ++i) off_a[i] = (uint32_t)min((wave * LA + i) * RPL + lane / PIECES, g.m - 1 - m0) * (uint32_t)g.lda;
  auto exchanged = [](int row, int p) { return KB == 128 ? p ^ (row / 2 % 8) : p ^ (row % 16); };
  const int stages = (g.k + KB - 1) / KB;
  // Direct load number i of the wave's LW + LA of a stage.  Loads of stages that
  // do not exist read an empty buffer, so that every stage counts the same
  // number of loads.
  auto fetch = [&](int stage, int8_t *buf, int i) {
    const int k0 = stage * KB;
    const uint32_t bytes = __builtin_amdgcn_readfirstlane(stage < stages ? -1 : 0);
    const int j = i < LW ? wave * LW + i : wave * LA + i - LW;
    // the lane's piece: the exchange repeats after PERIOD direct loads
    const uint32_t at = min(exchanged(j % PERIOD * RPL + lane / PIECES, lane % PIECES) * 16, last - k0);
    FB_LDS int8_t *dst = (FB_LDS int8_t *)buf + j * 1024;
    if (i < LW) load_to_lds(buffer_of(base_w, bytes), off_w[i] + at, k0, dst);
    else load_to_lds(buffer_of(base_a, bytes), off_a[i - LW] + at, k0, dst + BN * KB);
  };
  auto fetch_stage = [&](int stage, int8_t *buf) {
#pragma unroll
    for (int i = 0; i < LW + LA; ++i) fetch(stage, buf, i);
  };
  auto piece_at = [&](int8_t *buf, int row, int p) {
    return reinterpret_cast<i32x4 *>(buf + row * KB + exchanged(row, p) * 16);
  };
  // Where k ends inside a stage, the tokens' pieces behind it are cleared (what
  // the weights hold there is multiplied with these zeros).
  auto clear_tail = [&](int8_t *buf) {
    const int left = g.k - (stages - 1) * KB;
    for (int i = threadIdx.x; i < BM * PIECES; i += 64 * W) {
      const int p = i % PIECES;
      i32x4 *at = piece_at(buf, BN + i / PIECES, p);
      if (p * 16 + 16 > left) *at = mask_tail(*at, p * 16, left);
    }
  };
  const int wk = wave % WK, wm = wave / WK % WM, wn = wave / WK / WM;
  const int r = lane % 32, half = lane / 32;
  i32x16 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x16{};
  i32x4 wv[2][G][NT], av[2][G][MT];
  auto load_step = [&](int8_t *buf, int s, int set) {
#pragma unroll
    for (int b = 0; b < G; ++b) {
      const int p = 2 * (wk * BLOCKS + s * G + b) + half;
#pragma unroll
      for (int i = 0; i < NT; ++i) wv[set][b][i] = *piece_at(buf, (wn * NT + i) * 32 + r, p);
#pragma unroll
      for (int j = 0; j < MT; ++j) av[set][b][j] = *piece_at(buf, BN + (wm * MT + j) * 32 + r, p);
    }
  };
  auto multiply = [&](int set) {
#pragma unroll
    for (int b = 0; b < G; ++b)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[set][b][i], av[set][b][j], acc[i][j], 0, 0, 0);
  };
  // The products of a step with a stage's loads between them: all loads at once
  // would hold the wave until the memory pipe has taken them.
  auto multiply_and_fetch = [&](int set, int stage, int8_t *buf) {
    constexpr int PRODUCTS = G * NT * MT, L = LW + LA;
#pragma unroll
    for (int x = 0; x < PRODUCTS; ++x) {
      const int b = x / (NT * MT), i = x / MT % NT, j = x % MT;
#pragma unroll
      for (int l = x * L / PRODUCTS; l < (x + 1) * L / PRODUCTS; ++l) fetch(stage, buf, l);
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[set][b][i], av[set][b][j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // One stage that another follows; its first step's fragments are in set
  // `first`.  All reads of a step stand before the products of the step before,
  // and the barrier that ends the stage's reads (and tells that the next stage
  // has landed: the loads of S - 2 later ones may be in flight) before the last
  // step's products, which cover the first reads and the loads behind it.
  auto run_stage = [&](int t, int8_t *cur, int8_t *nxt, int first) {
#pragma unroll
    for (int s = 0; s + 1 < STEPS; ++s) {
      load_step(cur, s + 1, (first + s + 1) % 2);
      multiply((first + s) % 2);
      __builtin_amdgcn_sched_group_barrier(0x100, G * (NT + MT), 0);  // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x008, G * NT * MT, 0);    // products
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_and_meet<(S - 2) * (LW + LA)>();
    if (t + 2 == stages && g.k % KB) {
      clear_tail(nxt);
      wait_and_meet<(S - 2) * (LW + LA)>();
    }
    load_step(nxt, 0, (first + STEPS) % 2);
    __builtin_amdgcn_sched_barrier(0);
    multiply_and_fetch((first + STEPS - 1) % 2, t + S, cur);
  };
#pragma unroll
  for (int i = 0; i < S; ++i) fetch_stage(i, lds + i * STAGE);
  wait_and_meet<(S - 1) * (LW + LA)>();
  if (stages == 1 && g.k % KB) {
    clear_tail(lds);
    wait_and_meet<(S - 1) * (LW + LA)>();
  }
  load_step(lds, 0, 0);
  int slot = 0, t = 0;
  auto go = [&](int first) {
    const int next = slot + 1 == S ? 0 : slot + 1;
    run_stage(t++, lds + slot * STAGE, lds + next * STAGE, first);
    slot = next;
  };
  if (STEPS % 2) {  // an odd number of steps: the sets take turns by stage
    while (t + 2 < stages) {
      go(0);
      go(1);
    }
    if (t + 1 < stages) {
      go(0);
#pragma unroll
      for (int b = 0; b < G; ++b) {
#pragma unroll
        for (int i = 0; i < NT; ++i) wv[0][b][i] = wv[1][b][i];
#pragma unroll
        for (int j = 0; j < MT; ++j) av[0][b][j] = av[1][b][j];
      }
    }
  } else {
    while (t + 1 < stages) go(0);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (s + 1 < STEPS) load_step(lds + slot * STAGE, s + 1, (s + 1) % 2);
    multiply(s % 2);
  }
  __builtin_amdgcn_s_waitcnt(0);  // no direct load is in flight when the workgroup ends
  if (WK > 1) {  // the waves of a tile add their sums (exact, in any order)
    wait_and_meet<0>();
    i32x16 *sums = reinterpret_cast<i32x16 *>(lds);  // the first sums_bytes of the stages' memory
    const int pair = (wn * WM + wm) * NT * MT;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        if (wk > 0) sums[((wk - 1) * WN * WM * NT * MT + pair + i * MT + j) * 64 + lane] = acc[i][j];
    wait_and_meet<0>();
    if (wk > 0) return;
#pragma unroll
    for (int v = 1; v < WK; ++v)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] += sums[((v - 1) * WN * WM * NT * MT + pair + i * MT + j) * 64 + lane];
  }
  // Outputs.  A lane holds four channels of one token at a time; stored as they
  // are, 32 rows would be touched 16 bytes each.  So a wave turns its tokens x 32 C
  // channels at a time in a piece of LDS of its own and stores up to 128
  // consecutive bytes of a row.
  typedef typename E::raw raw;
  constexpr int C = NT >= 2 && sizeof(raw) == 2 ? 2 : 1, COLS = 32 * C, PITCH = COLS + 16 / (int)sizeof(raw);
  constexpr int PER = 16 / (int)sizeof(raw), LANES = COLS / PER;  // channels of a 16-byte piece; pieces of a row
  constexpr int TILES = WN * WM, ROWS = 32 * MT;                  // wave tiles; tokens of one
  static_assert(NT % C == 0 && sums_bytes + TILES * ROWS * PITCH * (int)sizeof(raw) <= S * STAGE,
                "the turned tiles fit the stages' memory");
  if (WK == 1) wait_and_meet<0>();  // every wave has read its last fragments
  else __builtin_amdgcn_s_waitcnt(0);
  // (the addresses are not to be computed before the loop and held through it)
  int ne = n0 + wn * NT * 32, me = m0 + wm * ROWS;
  asm volatile("" : "+s"(ne), "+s"(me));
  raw *out = reinterpret_cast<raw *>(lds + sums_bytes) + (wn * WM + wm) * ROWS * PITCH;
  float sa[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) sa[j] = g.a_scale[(uint32_t)min(me + j * 32 + r, g.m - 1)];
#pragma unroll
  for (int i0 = 0; i0 < NT; i0 += C) {
    // lane l of a 32 x 32 tile holds token l % 32, channels 8 q + 4 (l / 32) .. + 3
#pragma unroll
    for (int i = i0; i < i0 + C; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const Channels c = load_channels(g, ne + i * 32 + 8 * q + 4 * half);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          raw v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = E::round((float)acc[i][j][4 * q + e] * sa[j] * c.scale[e] + c.bias[e]);
          put4(out + (j * 32 + r) * PITCH + (i - i0) * 32 + 8 * q + 4 * half, v);
        }
      }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < ROWS * LANES / 64; ++p) {
      const int row = (p * 64 + lane) / LANES, col = lane % LANES * PER;
      const i32x4 v = *reinterpret_cast<const i32x4 *>(out + row * PITCH + col);
      if (me + row < g.m) store_piece((raw *)g.y + (int64_t)(me + row) * g.ldy, ne + i0 * 32 + col, g.n, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace fluxbin
