// rope_kernels.hpp -- from the rows of a QKV product to rotated queries and
// entries of a paged cache.
//
// Mathematics.  A head's row x is normed, u = x w / sqrt(mean(x^2) + eps) (or
// u = x), and pair j of its first R elements is a complex number turned by the
// angle pos * f_j: (a + ib) e^{i pos f_j}.  An angle of a far position needs more
// than fp32: pos f_j / pi is taken in fp64, its whole turns removed there, and
// the rest, in [-1, 1] half turns, goes to sincospi in fp32.
//
// Memory-bound: every row is read and written once.  A wave takes one token and as
// many of its rows as its lanes hold; the rows are loaded first, the angles of the
// token, one per lane, computed meanwhile and handed over in LDS, without a barrier.
// A lane has two runs of C elements of a row, so that no pair crosses lanes: in
// `half` order the runs are the two halves' parts of C pairs, else they lie side by
// side.  C is 8 (16-byte accesses) where dim and rotary_dim are multiples of 16,
// else 4.
//
// MI355X: 8192 tokens of 64 + 2 x 8 heads of 128, normed (336 MB) 67 us = 5.0 TB/s;
// 4096 tokens of 32 + 2 x 32 heads (201 MB) 43 us = 4.7 TB/s; one token 3.0 us
// against 1.6 of an empty launch.  A wave that took all rows of its token, its angles
// computed once for all of them, was slower (78 and 46 us; with the next rows loaded
// ahead 72 and 45): more waves hide more of the chain of look-ups (sequence, length,
// page) that stands before a store.
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
  int32_t rot, runs;  // runs: waves to a token
  float eps, inv_dim, scale;
};

// Sum over the LPR lanes of a row, the same in all of them, in a fixed order.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  auto step = [](float x, int y) { return x + __builtin_bit_cast(float, y); };
#define FB_DPP(x, ctrl) __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xf, 0xf, true)
  v = step(v, FB_DPP(v, 0xB1));                  // quad_perm 1 0 3 2
  v = step(v, FB_DPP(v, 0x4E));                  // quad_perm 2 3 0 1
  if (LPR >= 8) v = step(v, FB_DPP(v, 0x141));   // the other half of eight lanes
  if (LPR >= 16) v = step(v, FB_DPP(v, 0x140));  // the other half of sixteen
#undef FB_DPP
  if (LPR >= 32) v += __shfl_xor(v, 16);
  return v;
}

// C elements as they are stored.
template <typename E, int C>
struct Run {
  typedef uint32_t words __attribute__((ext_vector_type(C / 2), aligned(2)));
  words w;
  __device__ __forceinline__ void read(const uint16_t *p) { w = *reinterpret_cast<const words *>(p); }
  __device__ __forceinline__ void write(uint16_t *p) const { *reinterpret_cast<words *>(p) = w; }
  __device__ __forceinline__ float get(int i) const { return E::load((uint16_t)(w[i / 2] >> (16 * (i % 2)))); }
  __device__ __forceinline__ void set(const float *f) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) w[i] = (uint32_t)E::round(f[2 * i]) | (uint32_t)E::round(f[2 * i + 1]) << 16;
  }
};

// One wave per token and run of 64 / LPR of its heads + 2 kv_heads rows (queries,
// keys, values); LPR lanes to a row; near: pairs (2j, 2j + 1).
template <typename E, int C, int LPR, bool NORM>
__global__ __launch_bounds__(256) void rope_append_kernel(const RopeArgs a, const bool near) {
  __shared__ float turns[4][256];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Paged &b = a.b;
  const int64_t id = (int64_t)blockIdx.x * 4 + wave;
  const int token = __builtin_amdgcn_readfirstlane((int)(id / a.runs));
  if (token >= b.tokens) return;
  const int queries = a.q ? b.heads : 0, c = lane % LPR;
  const int r = (int)(id % a.runs) * (64 / LPR) + lane / LPR;
  const bool query = r < queries, key = !query && r < queries + b.kv_heads;
  const bool live = r < queries + 2 * b.kv_heads && 2 * C * c < b.dim, turned = 2 * C * c < a.rot;
  // where the lane's two runs start
  const int e0 = turned && !near ? C * c : 2 * C * c, e1 = turned && !near ? a.rot / 2 + C * c : 2 * C * c + C;
  const uint16_t *src = query ? a.q + (int64_t)token * a.ldq + r * b.dim
                        : key ? a.k + (int64_t)token * a.ldk + (r - queries) * b.dim
                              : a.v + (int64_t)token * a.ldv + (r - queries - b.kv_heads) * b.dim;
  Run<E, C> lo, hi, w0, w1;
  lo.w = hi.w = 0;
  const uint16_t *norm = NORM && query ? a.q_norm : NORM && key ? a.k_norm : nullptr;
  if (live) {
    lo.read(src + e0);
    hi.read(src + e1);
    if (norm) {
      w0.read(norm + e0);
      w1.read(norm + e1);
    }
  }

  // whose row it is, and its index
  Found f{token, token, token + 1, 0};
  if (b.seq_starts) {
    f = find_sequence(b, lane, [&](int start, int) { return start <= token; });
    if (f.seq >= b.seqs || token < f.start) return;  // behind the last sequence, or before the first
  } else {
    f.len = b.kv_lens[token];
  }
  const int at = f.len - (f.next - f.start) + (token - f.start);
  const int page = at >= 0 ? page_of(b, f.seq, at) : -1;
  const int64_t place = (int64_t)page * b.page_stride + (int64_t)(at & ((1 << b.page_shift) - 1)) * b.token_stride;

  float cs[C], sn[C];
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
      for (int i = 0; i < C; ++i) {
        cs[i] = turns[wave][2 * (C * c + i)];
        sn[i] = turns[wave][2 * (C * c + i) + 1];
      }
    }
  }

  float v[2 * C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    v[i] = lo.get(i);
    v[C + i] = hi.get(i);
  }
  if (NORM) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * C; ++i) ss = fmaf(v[i], v[i], ss);
    ss = row_sum<LPR>(ss);
    if (norm && live) {
      const float inv = ss < __builtin_inff() ? 1.0f / sqrtf(fmaf(ss, a.inv_dim, a.eps)) : __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < C; ++i) {
        v[i] = v[i] * inv * w0.get(i);
        v[C + i] = v[C + i] * inv * w1.get(i);
      }
    }
  }
  if (query || key) {  // values are copied as they are stored
    if (turned) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float p = near ? v[2 * i] : v[i], s = near ? v[2 * i + 1] : v[C + i];
        const float re = p * cs[i] - s * sn[i], im = s * cs[i] + p * sn[i];
        v[near ? 2 * i : i] = re;
        v[near ? 2 * i + 1 : C + i] = im;
      }
    }
    lo.set(v);
    hi.set(v + C);
  }
  if (live && (query || page >= 0)) {
    uint16_t *dst = query ? a.q_out + (int64_t)token * a.ldqo + r * b.dim
                          : (key ? b.k : b.v) + place + (int64_t)(r - queries - (key ? 0 : b.kv_heads)) * b.head_stride;
    lo.write(dst + e0);
    hi.write(dst + e1);
  }
}

}  // namespace fluxbin
