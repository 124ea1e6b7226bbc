// rope_kernels.hpp -- from the rows of a QKV product to rotated queries and
// entries of a paged cache.
//
// Mathematics.  A head's row x is normed, u = x w / sqrt(mean(x^2) + eps) (or
// u = x), and pair j of its first R elements is a complex number turned by the
// angle pos * f_j: (a + ib) e^{i pos f_j}.  An angle of a far position needs more
// than fp32: pos f_j / pi is taken in fp64, its whole turns removed there, and
// the rest, in [-1, 1] half turns, goes to sincospi in fp32.
//
// Memory-bound: every row is read and written once.  A wave takes one token and
// some of its rows, so the angles of a token, one per lane, are computed once per
// wave, handed over in LDS and used for all its heads, without a barrier; the
// rows of a step are loaded before the angles are computed.  A row is dim / 8
// lanes of eight elements, the four pairs of a lane side by side in `near` order
// and two runs of four elements in `half` order, so that no pair crosses lanes.
#pragma once

#include "elements.hpp"
#include "paged_batch.hpp"

namespace fluxbin {

struct RopeArgs {
  Paged b;
  const uint16_t *q, *k, *v, *q_norm, *k_norm;  // q and the norms may be null
  uint16_t *q_out;
  const double *freq;
  const int32_t *positions;  // may be null: the index in the cache
  int64_t ldq, ldk, ldv, ldqo;
  int32_t rot, rows_per_wave;
  float eps, inv_dim, scale;
};

// Sum over the LPR lanes of a row, the same in all of them, in a fixed order.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  auto step = [](float x, int y) { return x + __builtin_bit_cast(float, y); };
#define FB_DPP(x, ctrl) __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xf, 0xf, true)
  v = step(v, FB_DPP(v, 0xB1));                  // quad_perm 1 0 3 2
  v = step(v, FB_DPP(v, 0x4E));                  // quad_perm 2 3 0 1
  v = step(v, FB_DPP(v, 0x141));                 // the other half of eight lanes
  if (LPR >= 16) v = step(v, FB_DPP(v, 0x140));  // the other half of sixteen
#undef FB_DPP
  if (LPR >= 32) v += __shfl_xor(v, 16);
  return v;
}

// One wave per token and run of rows_per_wave of its heads + 2 kv_heads rows
// (queries, keys, values); LPR lanes to a row, U steps of 64 / LPR rows in
// flight; near: pairs (2j, 2j + 1).
template <typename E, int LPR, int U, bool NORM>
__global__ __launch_bounds__(256) void rope_append_kernel(const RopeArgs a, const int runs, const bool near) {
  constexpr int RPS = 64 / LPR;  // rows of a step
  __shared__ float turns[4][256];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Paged &b = a.b;
  const int64_t id = (int64_t)blockIdx.x * 4 + wave;
  const int token = __builtin_amdgcn_readfirstlane((int)(id / runs)), run = (int)(id % runs);
  if (token >= b.tokens) return;
  const int queries = a.q ? b.heads : 0, rows = queries + 2 * b.kv_heads;
  const int from = run * a.rows_per_wave, to = min(from + a.rows_per_wave, rows);
  const int slot = lane / LPR, c = lane % LPR;
  const bool inside = 8 * c < b.dim, turned = 8 * c < a.rot;
  // elements 0 .. 3 and 4 .. 7 of the lane
  const int e0 = turned && !near ? 4 * c : 8 * c, e1 = turned && !near ? a.rot / 2 + 4 * c : 8 * c + 4;

  words2 x[U][2];
  const auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * RPS + slot;
      const uint16_t *p = r < queries ? a.q + (int64_t)token * a.ldq + r * b.dim
                          : r < queries + b.kv_heads ? a.k + (int64_t)token * a.ldk + (r - queries) * b.dim
                                                     : a.v + (int64_t)token * a.ldv + (r - queries - b.kv_heads) * b.dim;
      x[u][0] = x[u][1] = words2{0, 0};
      if (r < to && inside) {
        x[u][0] = *reinterpret_cast<const words2 *>(p + e0);
        x[u][1] = *reinterpret_cast<const words2 *>(p + e1);
      }
    }
  };
  load(from);

  // whose row it is, and its index
  int seq = token, at, n = 1, nth = 0;
  if (b.seq_starts) {
    if (token < b.seq_starts[0]) return;
    seq = count_starts(b.seqs, lane, [&](int j) { return b.seq_starts[j] <= token; });
    if (seq >= b.seqs) return;
    const int start = b.seq_starts[seq];
    n = b.seq_starts[seq + 1] - start;
    nth = token - start;
  }
  at = b.kv_lens[seq] - n + nth;
  const int page = at >= 0 ? page_of(b, seq, at) : -1;
  const int64_t place = (int64_t)page * b.page_stride + (int64_t)(at & ((1 << b.page_shift) - 1)) * b.token_stride;

  float cs[4], sn[4];
  {
    const double pos = (double)(a.positions ? a.positions[token] : at);
    for (int j = lane; j < a.rot / 2; j += 64) {
      const double t = pos * (a.freq[j] * 0.31830988618379067154);  // half turns
      float s, co;
      sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &co);
      turns[wave][2 * j] = co * a.scale;
      turns[wave][2 * j + 1] = s * a.scale;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = turns[wave][8 * c + 2 * i];
        sn[i] = turns[wave][8 * c + 2 * i + 1];
      }
    }
  }

  for (int base = from; base < to; base += RPS * U) {
    if (base != from) load(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * RPS + slot;
      const bool query = r < queries, key = !query && r < queries + b.kv_heads, live = r < to && inside;
      words2 lo = x[u][0], hi = x[u][1];
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = E::load((uint16_t)(lo[i / 2] >> (16 * (i % 2))));
        f[4 + i] = E::load((uint16_t)(hi[i / 2] >> (16 * (i % 2))));
      }
      if (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
        ss = row_sum<LPR>(ss);
        const uint16_t *w = query ? a.q_norm : key ? a.k_norm : nullptr;
        if (w && live) {
          const float inv = ss < __builtin_inff() ? 1.0f / sqrtf(fmaf(ss, a.inv_dim, a.eps)) : __builtin_nanf("");
          const words2 w0 = *reinterpret_cast<const words2 *>(w + e0), w1 = *reinterpret_cast<const words2 *>(w + e1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = f[i] * inv * E::load((uint16_t)(w0[i / 2] >> (16 * (i % 2))));
            f[4 + i] = f[4 + i] * inv * E::load((uint16_t)(w1[i / 2] >> (16 * (i % 2))));
          }
        }
      }
      if (turned && (query || key)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = near ? f[2 * i] : f[i], s = near ? f[2 * i + 1] : f[4 + i];
          const float re = p * cs[i] - s * sn[i], im = s * cs[i] + p * sn[i];
          if (near) {
            f[2 * i] = re;
            f[2 * i + 1] = im;
          } else {
            f[i] = re;
            f[4 + i] = im;
          }
        }
      }
      if (query || key) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lo[i] = (uint32_t)E::round(f[2 * i]) | (uint32_t)E::round(f[2 * i + 1]) << 16;
          hi[i] = (uint32_t)E::round(f[4 + 2 * i]) | (uint32_t)E::round(f[5 + 2 * i]) << 16;
        }
      }
      if (live && (query || page >= 0)) {
        uint16_t *p = query ? a.q_out + (int64_t)token * a.ldqo + r * b.dim
                            : (key ? b.k : b.v) + place + (int64_t)(r - queries - (key ? 0 : b.kv_heads)) * b.head_stride;
        *reinterpret_cast<words2 *>(p + e0) = lo;
        *reinterpret_cast<words2 *>(p + e1) = hi;
      }
    }
  }
}

}  // namespace fluxbin
