// attention_kernels.hpp -- attention of new tokens over a paged cache.
//
// Mathematics.  With c = scale log2(e) and raw products s_j = q . k_j, a query's
// running maximum m (of the s_j seen) and
//     p_j = 2^(c s_j - c m + 7),  l = sum p_j,  o = sum p_j v_j,
// keys come in tiles; where a tile raises m, l and o are multiplied with
// 2^(c (m_old - m_new)).  out = o / l, lse = ln2 (c m - 7 + log2 l).  The factor 2^7
// keeps small weights out of fp16's subnormals.  Two sets of keys are joined in
// the same way, so keys may be split over waves and workgroups.
//
// All rows that read one key head are rows of one matrix: row r of a sequence is
// query head r % G of its group of G and token r / G.  Both products run
// transposed on v_mfma_f32_32x32x16, S^T = K Q^T and O^T = V^T P^T, so that a lane
// holds one query: maximum, sum and factors are a lane's own, but for one exchange
// with the lane 32 further, which holds the same query's other keys.  The
// registers in which S^T leaves the first product are the operand of the second
// as they are, if V^T is taken in the same order of keys, which the transposing
// LDS reads (four keys of a dimension each) give.
//
// Keys and values go from the cache's pages straight to LDS by groups of 16 keys
// (which no page divides), a row's 16-byte pieces exchanged by its number so that
// the fragment reads fall into all banks; rows that nobody sees read an empty part
// of the buffer and arrive as zeros, whatever the cache holds there.
#pragma once

#include "elements.hpp"
#include "lds_loads.hpp"
#include "paged_batch.hpp"
#include "wave_ops.hpp"

namespace fluxbin {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct AttentionArgs {
  Paged b;
  const uint16_t *q;
  uint16_t *out;
  float *lse;      // may be null
  float *part;     // splits > 1: o of [row][split][dim], then (c m, l) of [row][split]
  int64_t ldq, ldo, parts;  // parts: tokens * heads * splits
  int32_t group, window, splits, tiles;
  float c;
};

constexpr float kWeightShift = 7.0f;

template <typename E>
__device__ __forceinline__ f32x16 multiply(u32x4 a, u32x4 b, f32x16 acc);
template <>
__device__ __forceinline__ f32x16 multiply<F16>(u32x4 a, u32x4 b, f32x16 acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 multiply<BF16>(u32x4 a, u32x4 b, f32x16 acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}

// Two values rounded to nearest even, the first in the low half.
template <typename E>
__device__ __forceinline__ uint32_t pair_of(float x, float y) {
  return (uint32_t)E::round(x) | (uint32_t)E::round(y) << 16;
}

// A lane's value and that of the lane 32 away, the lower lane's first.  The second
// operand is made a value of its own: of one value given twice the compiler takes
// both results to be the same.
struct Halves {
  float lo, hi;
};
__device__ __forceinline__ Halves both_halves(float v) {
  int x = __builtin_bit_cast(int, v), y = x;
  asm("" : "+v"(y));
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  return Halves{__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1])};
}
__device__ __forceinline__ float other_half_max(float v) {
  const Halves h = both_halves(v);
  return fmaxf(h.lo, h.hi);
}
__device__ __forceinline__ float other_half_sum(float v) {
  const Halves h = both_halves(v);
  return h.lo + h.hi;
}

// A row of D elements in LDS is D / 8 pieces of 16 bytes, at places exchanged by
// the row's number: K's fragment reads take one piece of 16 consecutive rows at
// once, V's 64 bytes of four consecutive ones, and both then fill all 64 banks.
template <int D>
__device__ __forceinline__ int k_place(int row, int piece) {
  return piece ^ (D == 64 ? row / 2 % 8 : row % 16);
}
template <int D>
__device__ __forceinline__ int v_place(int row, int piece) {
  return piece ^ (D == 64 ? 4 * (row / 2 % 2) : 4 * (row % 4));
}

// The rows that a workgroup has: BM rows of one sequence and key head.
struct Rows {
  int seq, first, count;     // first row of the sequence's rows; the sequence's rows (0: nothing to do)
  int start, before;         // first token of the sequence; its index in the cache
  int p_lo, p_hi;            // indices of the first and last token here
  int lo, hi;                // keys that some row sees, [lo, hi)
};

template <int BM>
__device__ __forceinline__ Rows rows_of(const AttentionArgs &a, int tile, int lane) {
  const Paged &b = a.b;
  Rows r{};
  // Tile numbers of sequence s start at floor(start * G / BM) + s, which leaves
  // every sequence at least the tiles that its rows fill.
  const auto first_tile = [&](int s) { return (int)((int64_t)row_start(b, s) * a.group / BM) + s; };
  r.seq = count_starts(b.seqs, lane, [&](int s) { return first_tile(s) <= tile; });
  if (r.seq >= b.seqs) return r;
  r.start = row_start(b, r.seq);
  const int n = row_start(b, r.seq + 1) - r.start;
  r.first = (tile - first_tile(r.seq)) * BM;
  if (n <= 0 || r.first < 0 || r.first >= n * a.group) return r;
  r.count = n * a.group;
  const int len = b.kv_lens[r.seq], given = b.seq_starts ? b.seq_starts[r.seq + 1] - b.seq_starts[r.seq] : 1;
  r.before = len - given + (b.seq_starts ? r.start - b.seq_starts[r.seq] : 0);
  r.p_lo = r.before + r.first / a.group;
  r.p_hi = r.before + (min(r.first + BM, r.count) - 1) / a.group;
  r.hi = max(0, min(r.p_hi, (b.table_pages << b.page_shift) - 1) + 1);
  r.lo = a.window ? max(0, r.p_lo - a.window + 1) : 0;
  return r;
}

// One group of 16 keys on its way to LDS: where it comes from and which of its
// rows count.
struct Group {
  const int8_t *base;
  uint32_t bytes;
  int first;
};

// key0: the group's first index, a multiple of 16; page: its page or -1.
__device__ __forceinline__ Group group_of(const Paged &b, const uint16_t *cache, int head, int key0, int page, const Rows &r) {
  Group g;
  const int last = min(r.hi - key0, 16);
  g.first = r.lo - key0;
  g.base = in_scalars(reinterpret_cast<const int8_t *>(cache + (int64_t)max(page, 0) * b.page_stride + (int64_t)head * b.head_stride +
                                                       (int64_t)(key0 & ((1 << b.page_shift) - 1)) * b.token_stride));
  g.bytes = __builtin_amdgcn_readfirstlane(page >= 0 && last > 0 ? (uint32_t)(((last - 1) * b.token_stride + b.dim) * 2) : 0u);
  return g;
}

constexpr uint32_t kNowhere = 0x7ffffff0u;  // an offset beyond every buffer: zeros

// Loads of a group: D / 32 of 1 KiB, each 512 / D rows; `off`: each lane's offsets.
template <int D>
struct GroupLoads {
  static constexpr int kLoads = D / 32, kRows = 512 / D;
  static __device__ __forceinline__ void offsets(const Paged &b, int lane, bool value, uint32_t (&off)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kRows + lane / (D / 8), place = lane % (D / 8);
      const int piece = value ? v_place<D>(row, place) : k_place<D>(row, place);
      off[i] = piece * 8 < b.dim ? (uint32_t)(row * b.token_stride * 2 + piece * 16) : kNowhere;
    }
  }
  static __device__ __forceinline__ void load(const Group &g, int lane, const uint32_t (&off)[kLoads], FB_LDS int8_t *dst) {
    const __amdgpu_buffer_rsrc_t from = buffer_of(g.base, g.bytes);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kRows + lane / (D / 8);
      load_to_lds(from, g.first > 0 && row < g.first ? kNowhere : off[i], 0, dst + i * 1024);
    }
  }
};

// A wave's 32 x QB queries against a tile of KT keys.
template <typename E, int D, int QB, int KT>
struct WaveTile {
  static constexpr int KB = KT / 32, STEPS = D / 16, DB = D / 32;
  u32x4 q[QB][STEPS];
  f32x16 o[DB][QB];
  float m[QB], l[QB];     // m: largest s so far; l: this lane's part of the sum
  int p[QB], from[QB];    // the query's index and the first that it sees

  __device__ __forceinline__ void start(const AttentionArgs &a, const Rows &r, int head, int row0, int lane) {
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      const int row = r.first + row0 + x * 32 + lane % 32;
      const bool live = row < r.count;
      const int token = row / a.group;
      const uint16_t *src = a.q + (int64_t)(r.start + token) * a.ldq + (head * a.group + row % a.group) * a.b.dim;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int d = 16 * s + 8 * (lane / 32);
        q[x][s] = u32x4{0, 0, 0, 0};
        if (live && d < a.b.dim) {
          const words4 v = *reinterpret_cast<const words4 *>(src + d);
          q[x][s] = u32x4{v[0], v[1], v[2], v[3]};
        }
      }
      m[x] = -__builtin_inff();
      l[x] = 0.0f;
      p[x] = live ? r.before + token : -1;
      from[x] = a.window ? max(0, p[x] - a.window + 1) : 0;
#pragma unroll
      for (int i = 0; i < DB; ++i) o[i][x] = f32x16{};
    }
  }

  // there: bit g says that the tile's group g of 16 keys has a page; all of them
  // and no border of anybody's view inside the tile: masked = false.  mixed: the
  // tile has keys that some rows see and others do not.
  __device__ __forceinline__ void take(const AttentionArgs &a, const int8_t *kt, const int8_t *vt, int key0, bool masked, bool mixed,
                                       uint32_t there, int lane) {
    const int half = lane / 32;
    f32x16 s[KB][QB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
#pragma unroll
      for (int x = 0; x < QB; ++x) s[k][x] = f32x16{};
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int row = 32 * k + lane % 32;
        const u32x4 f = *reinterpret_cast<const u32x4 *>(kt + row * D * 2 + k_place<D>(row, 2 * i + half) * 16);
#pragma unroll
        for (int x = 0; x < QB; ++x) s[k][x] = multiply<E>(f, q[x][i], s[k][x]);
      }
    }
    if (masked) {
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int x = 0; x < QB; ++x)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + 32 * k + 8 * (i / 4) + 4 * half + i % 4;
            const bool seen = key >= from[x] && key <= p[x] && (there >> (2 * k + i / 8) & 1);
            s[k][x][i] = seen ? s[k][x][i] : -__builtin_inff();
          }
    }
    u32x4 w[KB][2][QB];  // the weights, 16 keys to an operand
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      float top = s[0][x][0];
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[k][x][i]);
      top = fmaxf(m[x], other_half_max(top));
      const float base = top == -__builtin_inff() ? 0.0f : top;
      const float factor = __builtin_amdgcn_exp2f((m[x] - base) * a.c), shift = kWeightShift - base * a.c;
      m[x] = top;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[k][x][i] = __builtin_amdgcn_exp2f(fmaf(s[k][x][i], a.c, shift));
          sum += s[k][x][i];
        }
      l[x] = fmaf(l[x], factor, sum);
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) w[k][j][x][i] = pair_of<E>(s[k][x][8 * j + 2 * i], s[k][x][8 * j + 2 * i + 1]);
#pragma unroll
      for (int i = 0; i < DB; ++i) o[i][x] *= factor;
    }
    if (mixed && unclean(vt, lane)) {
      one_by_one(vt, w, lane);
      return;
    }
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          const u32x4 v = values(vt, 32 * k + 16 * j, i, lane);
#pragma unroll
          for (int x = 0; x < QB; ++x) o[i][x] = multiply<E>(v, w[k][j][x], o[i][x]);
        }
  }

  // V^T of dimensions 32 i .. + 31 and 16 keys in the order of the weights: lane l
  // has dimension l % 32 and the keys 4 (l / 32) + 0 .. 3, 8 + 4 (l / 32) + 0 .. 3.
  static __device__ __forceinline__ u32x4 values(const int8_t *vt, int key, int i, int lane) {
    u32x4 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = key + 8 * h + 4 * (lane / 32) + lane % 16 / 4;
      const int piece = 4 * i + lane / 16 % 2 * 2 + lane % 4 / 2;
      const int8_t *at = vt + row * D * 2 + v_place<D>(row, piece) * 16 + lane % 2 * 8;
      const s16x4 f = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FB_LDS s16x4 *)at);
      const u32x2 t = __builtin_bit_cast(u32x2, f);
      v[2 * h] = t[0];
      v[2 * h + 1] = t[1];
    }
    return v;
  }

  // Whether the tile holds a value that times 0 is not 0.
  static __device__ __forceinline__ bool unclean(const int8_t *vt, int lane) {
    constexpr uint32_t e = __is_same(E, F16) ? 0x7c00u : 0x7f80u;
    bool bad = false;
    for (int at = lane * 16; at < KT * D * 2; at += 1024) {
      const u32x4 v = *reinterpret_cast<const u32x4 *>(vt + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) bad = bad || (v[i] & e) == e || (v[i] >> 16 & e) == e;
    }
    return __any(bad);
  }

  // The second product where such values stand among keys that not every row
  // sees: key by key, a row leaving out those whose weight is 0.
  __device__ __forceinline__ void one_by_one(const int8_t *vt, const u32x4 (&w)[KB][2][QB], int lane) {
#pragma unroll 1
    for (int key = 0; key < KT; ++key) {
      const int hold = key / 4 % 2;  // which half of the wave has its weights, and where
      const int pick = key / 32 * 16 + key % 32 / 8 * 4 + key % 4;
#pragma unroll
      for (int x = 0; x < QB; ++x) {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < KB * 8; ++i) word = pick / 2 == i ? w[i / 8][i / 4 % 2][x][i % 4] : word;
        word = __shfl(word, lane % 32 + 32 * hold);
        const float f = E::load((uint16_t)(word >> (16 * (pick % 2))));
        if (f != 0.0f) {
#pragma unroll
          for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const u32x2 v = *reinterpret_cast<const u32x2 *>(vt + key * D * 2 + v_place<D>(key, 4 * i + j) * 16 + lane / 32 * 8);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[i][x][4 * j + e] = fmaf(f, E::load((uint16_t)(v[e / 2] >> (16 * (e % 2)))), o[i][x][4 * j + e]);
            }
        }
      }
    }
  }
};

// What a row comes to: its output and lse, or the part of a split.  v: elements
// d .. d + 3 of o.
__device__ __forceinline__ float lse_of(float cm, float l) {
  return l == 0.0f ? -__builtin_inff() : 0.69314718055994530942f * (cm - kWeightShift + log2f(l));
}
template <typename E>
__device__ __forceinline__ void put_out(const AttentionArgs &a, int64_t token, int head, int d, f32x4 v, float inv) {
  *reinterpret_cast<words2 *>(a.out + token * a.ldo + head * a.b.dim + d) =
      words2{pair_of<E>(v[0] * inv, v[1] * inv), pair_of<E>(v[2] * inv, v[3] * inv)};
}

// 128 x QB rows, 32 x QB to each of four waves, over one split of their keys; a
// workgroup's tiles of KT keys come by two buffers, the next one loaded while one is
// worked on.
template <typename E, int D, int QB>
__global__ __launch_bounds__(256) void attention_chunk_kernel(const AttentionArgs a) {
  constexpr int BM = 128 * QB, KT = D == 256 ? 32 : 64, GROUPS = KT / 16, JOBS = 2 * GROUPS / 4, BYTES = KT * D * 2;
  typedef GroupLoads<D> Loads;
  __shared__ __align__(1024) int8_t lds[2][2][BYTES];  // [buffer][K, V]
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Paged &b = a.b;
  // key heads go to the XCDs in turn, so that the workgroups that share one's
  // keys share an L2; the last tiles, which see most, start first
  const int head = blockIdx.x % b.kv_heads, rest = blockIdx.x / b.kv_heads;
  const int split = rest % a.splits, tile = a.tiles - 1 - rest / a.splits;
  const Rows r = rows_of<BM>(a, tile, lane);
  if (r.count == 0) return;

  const int begin = r.lo / KT, all = max(0, (r.hi + KT - 1) / KT - begin), per = (all + a.splits - 1) / a.splits;
  const int t0 = begin + min(split * per, all), t1 = begin + min((split + 1) * per, all);
  WaveTile<E, D, QB, KT> w;
  w.start(a, r, head, wave * 32 * QB, lane);

  uint32_t off[JOBS][Loads::kLoads];
#pragma unroll
  for (int j = 0; j < JOBS; ++j) Loads::offsets(b, lane, (j * 4 + wave) / GROUPS, off[j]);
  // lane g of `pages`: the page of the group g of the tile that is fetched next
  int pages;
  const auto find_pages = [&](int t) { pages = t < t1 ? page_of(b, r.seq, t * KT + 16 * (lane % GROUPS)) : -1; };
  const auto there_of = [&]() { return (uint32_t)__ballot(pages >= 0) & ((1u << GROUPS) - 1); };
  const auto fetch = [&](int t, int buf) {
#pragma unroll
    for (int j = 0; j < JOBS; ++j) {
      const int job = j * 4 + wave, g = job % GROUPS;
      const bool value = job / GROUPS;
      Loads::load(group_of(b, value ? b.v : b.k, head, t * KT + 16 * g, __builtin_amdgcn_readlane(pages, g), r), lane, off[j],
                  (FB_LDS int8_t *)lds[buf][value] + g * 16 * D * 2);
    }
  };
  find_pages(t0);
  uint32_t there = there_of();
  if (t0 < t1) fetch(t0, 0);
  find_pages(t0 + 1);
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) % 2;
    wait_and_meet<0>();
    const uint32_t next = there_of();
    if (t + 1 < t1) fetch(t + 1, buf ^ 1);
    find_pages(t + 2);
    const int key0 = t * KT;
    const bool border = key0 + KT - 1 > r.p_lo || (a.window && key0 <= r.p_hi - a.window);
    w.take(a, lds[buf][0], lds[buf][1], key0, border || there != (1u << GROUPS) - 1 || key0 + KT > r.hi, border && r.p_lo != r.p_hi,
           there, lane);
    there = next;
  }

#pragma unroll
  for (int x = 0; x < QB; ++x) {
    const int row = r.first + (wave * QB + x) * 32 + lane % 32;
    if (row >= r.count) continue;
    const float l = other_half_sum(w.l[x]), cm = w.m[x] * a.c;
    const int64_t token = r.start + row / a.group;
    const int h = head * a.group + row % a.group;
    const int64_t at = (token * b.heads + h) * a.splits + split;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (lane < 32) {
      if (a.splits > 1) {
        a.part[a.parts * b.dim + 2 * at] = cm;
        a.part[a.parts * b.dim + 2 * at + 1] = l;
      } else if (a.lse) {
        a.lse[token * b.heads + h] = lse_of(cm, l);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * i + 8 * j + 4 * (lane / 32);
        const f32x4 v{w.o[i][x][4 * j], w.o[i][x][4 * j + 1], w.o[i][x][4 * j + 2], w.o[i][x][4 * j + 3]};
        if (d < b.dim) {
          if (a.splits > 1) *reinterpret_cast<f32x4 *>(a.part + at * b.dim + d) = v;
          else put_out<E>(a, token, h, d, v, inv);
        }
      }
  }
}

// Up to 32 rows: the waves share them and split the keys, each with a ring of
// tiles of its own, so that nothing waits for another wave before the end.
template <int D>
struct Few {
  static constexpr int W = D == 256 ? 2 : 4, STAGES = 2, KT = 32, BYTES = KT * D * 2;
};
template <typename E, int D>
__global__ __launch_bounds__(64 * Few<D>::W) void attention_few_kernel(const AttentionArgs a) {
  typedef Few<D> F;
  constexpr int W = F::W, S = F::STAGES, KT = F::KT, BYTES = F::BYTES;
  typedef GroupLoads<D> Loads;
  constexpr int ROW = D + 4;  // floats of a row of the joined sums: rows four banks apart
  static_assert(W * 32 * ROW * 4 <= W * S * 2 * BYTES, "the waves' sums take the place of the tiles");
  __shared__ __align__(1024) int8_t lds[W * S * 2 * BYTES];
  __shared__ float stats[2][W][32];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Paged &b = a.b;
  const int head = blockIdx.x % b.kv_heads, rest = blockIdx.x / b.kv_heads;
  const int split = rest % a.splits, tile = rest / a.splits;
  const Rows r = rows_of<32>(a, tile, lane);
  if (r.count == 0) return;

  const int begin = r.lo / KT, all = max(0, (r.hi + KT - 1) / KT - begin), per = (all + a.splits - 1) / a.splits;
  const int t0 = begin + min(split * per, all), t1 = begin + min((split + 1) * per, all);
  WaveTile<E, D, 1, KT> w;
  w.start(a, r, head, 0, lane);

  uint32_t off_k[Loads::kLoads], off_v[Loads::kLoads];
  Loads::offsets(b, lane, false, off_k);
  Loads::offsets(b, lane, true, off_v);
  int8_t *mine = lds + wave * S * 2 * BYTES;
  // lane 2 i + g of `pages`: the page of the group g of the wave's tile number i
  // after the last look-up, made every 32 tiles
  int pages = -1;
  uint32_t there[S];
  // The wave's tile number n.  Loads of tiles that do not exist read an empty
  // buffer, so that every stage counts the same number of loads.
  const auto fetch = [&](int n, int stage) {
    if (n % 32 == 0) {
      const int t = t0 + wave + (n + lane / 2) * W;
      pages = t < t1 ? page_of(b, r.seq, t * KT + 16 * (lane % 2)) : -1;
    }
    const int t = t0 + wave + n * W;
    int8_t *dst = mine + stage * 2 * BYTES;
    there[stage] = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int page = __builtin_amdgcn_readlane(pages, n % 32 * 2 + g);
      there[stage] |= (uint32_t)(page >= 0) << g;
      Loads::load(group_of(b, b.k, head, t * KT + 16 * g, page, r), lane, off_k, (FB_LDS int8_t *)dst + g * 16 * D * 2);
      Loads::load(group_of(b, b.v, head, t * KT + 16 * g, page, r), lane, off_v, (FB_LDS int8_t *)dst + BYTES + g * 16 * D * 2);
    }
  };
  const auto work = [&](int t, int stage) {
    const int key0 = t * KT;
    const int8_t *from = mine + stage * 2 * BYTES;
    const bool border = key0 + KT - 1 > r.p_lo || (a.window && key0 <= r.p_hi - a.window);
    w.take(a, from, from + BYTES, key0, border || there[stage] != 3 || key0 + KT > r.hi, border && r.p_lo != r.p_hi, there[stage],
           lane);
  };
#pragma unroll
  for (int i = 0; i < S; ++i) fetch(i, i);
  for (int n = 0; t0 + wave + n * W < t1; n += S) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      wait_for_loads<(S - 1) * 4 * Loads::kLoads>();
      const int t = t0 + wave + (n + i) * W;
      if (t < t1) work(t, i);
      wait_for_reads();
      fetch(n + S + i, i);
    }
  }

  // Join the waves.
  const float l = other_half_sum(w.l[0]);
  wait_and_meet<0>();
  if (lane < 32) {
    stats[0][wave][lane] = w.m[0];
    stats[1][wave][lane] = l;
  }
  __syncthreads();
  const int mine_row = lane % 32;
  float top = -__builtin_inff();
#pragma unroll
  for (int v = 0; v < W; ++v) top = fmaxf(top, stats[0][v][mine_row]);
  const float factor = w.m[0] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((w.m[0] - top) * a.c);
  float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4 *>(sums + (wave * 32 + mine_row) * ROW + 32 * i + 8 * j + 4 * (lane / 32)) =
          f32x4{w.o[i][0][4 * j], w.o[i][0][4 * j + 1], w.o[i][0][4 * j + 2], w.o[i][0][4 * j + 3]} * factor;
  __syncthreads();
  const int rows = min(32, r.count - r.first);
  for (int x = threadIdx.x; x < rows * (D / 4); x += 64 * W) {
    const int row = x / (D / 4), d = x % (D / 4) * 4;
    if (d >= b.dim) continue;
    float big = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int v = 0; v < W; ++v) big = fmaxf(big, stats[0][v][row]);
    f32x4 o{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const float m = stats[0][v][row];
      if (m == -__builtin_inff()) continue;
      sum = fmaf(stats[1][v][row], __builtin_amdgcn_exp2f((m - big) * a.c), sum);
      o += *reinterpret_cast<const f32x4 *>(sums + (v * 32 + row) * ROW + d);
    }
    const int64_t token = r.start + (r.first + row) / a.group;
    const int h = head * a.group + (r.first + row) % a.group;
    const int64_t at = (token * b.heads + h) * a.splits + split;
    if (a.splits > 1) {
      *reinterpret_cast<f32x4 *>(a.part + at * b.dim + d) = o;
      if (d == 0) {
        a.part[a.parts * b.dim + 2 * at] = big * a.c;
        a.part[a.parts * b.dim + 2 * at + 1] = sum;
      }
    } else {
      put_out<E>(a, token, h, d, o, sum == 0.0f ? 0.0f : 1.0f / sum);
      if (a.lse && d == 0) a.lse[token * b.heads + h] = lse_of(big * a.c, sum);
    }
  }
}

// The parts of a row's splits joined, a wave to a row.
template <typename E>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttentionArgs a) {
  const Paged &b = a.b;
  const int lane = threadIdx.x % 64;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (row >= (int64_t)b.tokens * b.heads) return;
  const int token = (int)(row / b.heads);
  if (b.seq_starts && (token < b.seq_starts[0] || token >= b.seq_starts[b.seqs])) return;  // behind the last sequence
  float cm = -__builtin_inff(), l = 0.0f;
  if (lane < a.splits) {
    cm = a.part[a.parts * b.dim + 2 * (row * a.splits + lane)];
    l = a.part[a.parts * b.dim + 2 * (row * a.splits + lane) + 1];
  }
  const float top = wave_reduce<MaxF>(cm);
  const float f = cm == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(cm - top);
  const float sum = wave_reduce<SumF>(f == 0.0f ? 0.0f : f * l);
  f32x4 o{0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s) {
    const float fs = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), s));
    if (fs != 0.0f && 4 * lane < b.dim) o += *reinterpret_cast<const f32x4 *>(a.part + (row * a.splits + s) * b.dim + 4 * lane) * fs;
  }
  if (4 * lane < b.dim) put_out<E>(a, token, (int)(row % b.heads), 4 * lane, o, sum == 0.0f ? 0.0f : 1.0f / sum);
  if (a.lse && lane == 0) a.lse[row] = lse_of(top, sum);
}

}  // namespace fluxbin
