// attention_kernels.hpp -- attention of new tokens over a paged cache.
//
// Mathematics.  With c = scale log2(e) and raw products s_j = q . k_j, a query's
// running maximum m (of the s_j seen) and
//     p_j = 2^(c s_j - c m + 7),  l = sum p_j,  o = sum p_j v_j,
// keys come in tiles; where a tile raises m, l and o are multiplied with
// 2^(c (m_old - m_new)).  out = o / l, lse = ln2 (c m - 7 + log2 l).  m is raised only
// when a score passes it by more than kSlack (in powers of two), so weights reach
// 2^15; the factor 2^7 keeps small ones out of fp16's subnormals.  Weights are
// rounded to the activation type for the second product alone: l, and with it lse,
// is the fp32 sum of the weights before that.  That rounding of every weight adds
// about as much to an output's error as the output's own (in quadrature); a chunk's
// products are what bounds it and bear no more, single tokens wait for memory and
// take a second product with what the rounding left.  Two sets of keys are joined by
// moving both to the larger m, so keys may be split over waves and workgroups.
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
#include "key_weight.hpp"
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
  float *part, *stats;  // parts of rows: o [part][dim], (m, l) [part]
  int32_t *before;      // balanced: key tiles of the row tiles before each, and of all of them
  int64_t ldq, ldo;
  int32_t group, window, splits, tiles, workgroups;
  float c;
};

constexpr float kSlack = 8.0f;

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
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <typename E>
__device__ __forceinline__ uint32_t pair_of(float x, float y);
template <>
__device__ __forceinline__ uint32_t pair_of<F16>(float x, float y) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, f16x2));
}
template <>
__device__ __forceinline__ uint32_t pair_of<BF16>(float x, float y) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
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

// Tile numbers of sequence s start at floor(start * G / BM) + s, which leaves every
// sequence at least the tiles that its rows fill.  Starts are cut to the rows that
// exist.
template <int BM>
__device__ __forceinline__ int first_tile(const AttentionArgs &a, int start, int s) {
  return (int)((int64_t)max(0, min(start, a.b.tokens)) * a.group / BM) + s;
}

template <int BM>
__device__ __forceinline__ Rows rows_at(const AttentionArgs &a, int tile, const Found &f) {
  const Paged &b = a.b;
  Rows r{};
  r.seq = f.seq;
  if (r.seq >= b.seqs) return r;
  r.start = max(0, min(f.start, b.tokens));
  const int n = max(0, min(f.next, b.tokens)) - r.start;
  r.first = (tile - first_tile<BM>(a, f.start, r.seq)) * BM;
  if (n <= 0 || r.first < 0 || r.first >= n * a.group) return r;
  r.count = n * a.group;
  r.before = f.len - (f.next - f.start) + (r.start - f.start);
  r.p_lo = r.before + r.first / a.group;
  r.p_hi = r.before + (min(r.first + BM, r.count) - 1) / a.group;
  r.hi = max(0, min(r.p_hi, (b.table_pages << b.page_shift) - 1) + 1);
  r.lo = min(r.hi, a.window ? max(0, r.p_lo - a.window + 1) : 0);
  return r;
}

template <int BM>
__device__ __forceinline__ Rows rows_of(const AttentionArgs &a, int tile, int lane) {
  return rows_at<BM>(a, tile, find_sequence(a.b, lane, [&](int start, int s) { return first_tile<BM>(a, start, s) <= tile; }));
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
  template <bool ONCE>
  static __device__ __forceinline__ void load(const Group &g, int lane, const uint32_t (&off)[kLoads], FB_LDS int8_t *dst) {
    const __amdgpu_buffer_rsrc_t from = buffer_of(g.base, g.bytes);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * kRows + lane / (D / 8);
      load_to_lds<ONCE>(from, g.first > 0 && row < g.first ? kNowhere : off[i], 0, dst + i * 1024);
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

  typedef f32x16 Scores[KB][QB];  // S^T of a tile
  typedef u32x4 Weights[KB][2][QB];

  __device__ __forceinline__ void scores(const int8_t *kt, int lane, Scores &s) const {
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int x = 0; x < QB; ++x) s[k][x] = f32x16{};
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const int row = 32 * k + lane % 32;
        const u32x4 f = *reinterpret_cast<const u32x4 *>(kt + row * D * 2 + k_place<D>(row, 2 * i + lane / 32) * 16);
#pragma unroll
        for (int x = 0; x < QB; ++x) s[k][x] = multiply<E>(f, q[x][i], s[k][x]);
      }
  }

  // Scores to weights, which stay in s unrounded, with what that does to m, l and o.
  __device__ __forceinline__ void weights(float c, Scores &s, Weights &w) {
    float top[QB];
    bool rise = false;
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      top[x] = s[0][x][0];
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) top[x] = fmaxf(top[x], s[k][x][i]);
      top[x] = other_half_max(top[x]);
      rise = rise || (top[x] - m[x]) * c > kSlack || (m[x] == -__builtin_inff() && top[x] != m[x]);
    }
    if (__any(rise)) {
#pragma unroll
      for (int x = 0; x < QB; ++x) {
        const float up = fmaxf(m[x], top[x]);
        float factor = up == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((m[x] - up) * c);
        asm volatile("" : "+v"(factor));
        m[x] = up;
        l[x] *= factor;
#pragma unroll
        for (int i = 0; i < DB; ++i) o[i][x] *= factor;
      }
    }
#pragma unroll
    for (int x = 0; x < QB; ++x) {
      const float shift = m[x] == -__builtin_inff() ? 0.0f : kWeightShift - m[x] * c;
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = __builtin_amdgcn_exp2f(fmaf(s[k][x][8 * j + 2 * i], c, shift));
            const float b = __builtin_amdgcn_exp2f(fmaf(s[k][x][8 * j + 2 * i + 1], c, shift));
            s[k][x][8 * j + 2 * i] = a;
            s[k][x][8 * j + 2 * i + 1] = b;
            w[k][j][x][i] = pair_of<E>(a, b);
            sum[i % 2] += a + b;
          }
      l[x] += sum[0] + sum[1];
    }
  }

  // weights() with what its roundings leave, rounded in its turn, in `rest`.
  __device__ __forceinline__ void exact_weights(float c, Scores &s, Weights &w, Weights &rest) {
    weights(c, s, w);
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 0; x < QB; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = w[k][j][x][i];
            rest[k][j][x][i] = pair_of<E>(s[k][x][8 * j + 2 * i] - E::load((uint16_t)v), s[k][x][8 * j + 2 * i + 1] - E::load((uint16_t)(v >> 16)));
          }
  }

  __device__ __forceinline__ void add_values(const int8_t *vt, int lane, const Weights &w, const Weights *rest = nullptr) {
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          const u32x4 v = values(vt, 32 * k + 16 * j, i, lane);
#pragma unroll
          for (int x = 0; x < QB; ++x) {
            o[i][x] = multiply<E>(v, w[k][j][x], o[i][x]);
            if (rest) o[i][x] = multiply<E>(v, (*rest)[k][j][x], o[i][x]);
          }
        }
  }

  // Leaves out what a row does not see of the tile that begins at key0.  part: the
  // border of a row's view lies in it, or keys that are not there (bit g of `there`:
  // its group g of 16 has a page).  (The empty asm makes a value of the rare work
  // known there only, which keeps the compiler from doing that work always.)
  __device__ __forceinline__ void mask(Scores &s, bool part, int key0, uint32_t there, int lane) const {
    if (part) {
#pragma unroll
      for (int x = 0; x < QB; ++x) {
        // The lane's key 0 is number `mine`; keys lo .. lo + span behind it are seen,
        // one unsigned comparison each (lo out of reach: none).
        int mine = key0 + 4 * (lane / 32);
        asm volatile("" : "+v"(mine));
        const bool any = p[x] >= mine && from[x] <= p[x];
        const int lo = any ? max(from[x] - mine, 0) : 1 << 20;
        const uint32_t span = any ? (uint32_t)(p[x] - mine - lo) : 0;
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[k][x][i] = (uint32_t)(32 * k + 8 * (i / 4) + i % 4 - lo) <= span ? s[k][x][i] : -__builtin_inff();
        if (there != (1u << (2 * KB)) - 1) {
#pragma unroll
          for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[k][x][i] = there >> (2 * k + i / 8) & 1 ? s[k][x][i] : -__builtin_inff();
        }
      }
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

  // Whether an infinity or NaN has come into o: one among the values, which a weight
  // of 0 turns into NaN for rows that do not see it, or one among the scores; or
  // whether c m has left fp32's range, where the weights were not what they should be.
  __device__ __forceinline__ bool unclean(float c) const {
    float z = 0.0f;
#pragma unroll
    for (int x = 0; x < QB; ++x) z = m[x] == -__builtin_inff() ? z : fmaf(m[x] * c, 0.0f, z);
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int x = 0; x < QB; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) z = fmaf(o[i][x][e], 0.0f, z);
    return __any(!(z == 0.0f));
  }
};

// What a row comes to: its output and lse, or the part of a split.
__device__ __forceinline__ float lse_of(float m, float c, float l) {
  const float ln2 = 0.69314718055994530942f;  // before c, so that nothing passes lse itself
  return l == 0.0f ? -__builtin_inff() : fmaf(ln2 * m, c, ln2 * (log2f(l) - kWeightShift));
}
struct Place {
  uint16_t *out;
  float *part;  // null where the keys are not split
  float inv;
  template <typename E>
  __device__ __forceinline__ void put(int d, f32x4 o) const {
    if (part) *reinterpret_cast<f32x4 *>(part + d) = o;
    else *reinterpret_cast<words2 *>(out + d) = words2{pair_of<E>(o[0] * inv, o[1] * inv), pair_of<E>(o[2] * inv, o[3] * inv)};
  }
};

// Where a row's o goes: the output, or its part number `index` (< 0: none).  The
// row's lse, or the part's (m, l), is written here by the lane that is `first` of
// those that have the row.
__device__ __forceinline__ Place place_of(const AttentionArgs &a, const Rows &r, int head, int row, int64_t index, float m, float l, bool first) {
  const int token = r.start + row / a.group, h = head * a.group + row % a.group;
  Place p;
  p.out = a.out + (int64_t)token * a.ldo + h * a.b.dim;
  p.part = index >= 0 ? a.part + index * a.b.dim : nullptr;
  p.inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (first && index >= 0) {
    a.stats[2 * index] = m;
    a.stats[2 * index + 1] = l;
  } else if (first && a.lse) {
    a.lse[(int64_t)token * a.b.heads + h] = lse_of(m, a.c, l);
  }
  return p;
}

// The part that row x of a workgroup writes, where its first row writes part `parts`
// (< 0: none, the rows are whole).
__device__ __forceinline__ int64_t part_of(int64_t parts, int x) { return parts < 0 ? -1 : parts + x; }

// A sum of weighted values times a factor of 0 or more: an infinity or NaN in it, which
// has a weight above 0 however small, stays when the factor underflows.
__device__ __forceinline__ f32x4 rescaled(f32x4 o, float factor) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= fabsf(o[i]) < __builtin_inff() ? factor : 1.0f;
  return o;
}

// Rows [from, to) of a workgroup over the keys [k0, k1), one after the other by a
// wave: 64 keys at a time, a lane to a key, then a lane to four dimensions.  For
// rows that an infinity or NaN came into: a matrix product carries one to all its
// rows (0 times infinity); here a key that a row does not see, or whose score is
// -inf, is left out, and any other infinite value or NaN counts whatever its weight
// rounds to, so that neither the keys' order nor their division matters.
template <typename E>
__device__ __forceinline__ void rows_one_by_one(const AttentionArgs &a, const Rows &r, int head, int64_t parts, int from, int to, int step,
                                                int k0, int k1, int lane) {
  const Paged &b = a.b;
  for (int row = from; row < to; row += step) {
    const int token = row / a.group, p = r.before + token, first = a.window ? max(0, p - a.window + 1) : 0;
    const uint16_t *q = a.q + (int64_t)(r.start + token) * a.ldq + (head * a.group + row % a.group) * b.dim;
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 o{0, 0, 0, 0};
    for (int base = max(k0, first); base < min(k1, p + 1); base += 64) {
      const int key = base + lane;
      int page = -1;
      if (key < k1 && key <= p) page = page_of(b, r.seq, key);
      const int64_t at = page < 0 ? 0 : (int64_t)page * b.page_stride + (int64_t)head * b.head_stride +
                                            (int64_t)(key & ((1 << b.page_shift) - 1)) * b.token_stride;
      float s = -__builtin_inff();
      if (page >= 0) {
        s = 0.0f;
#pragma unroll 4
        for (int d = 0; d < b.dim; d += 8) {
          const words4 x = *reinterpret_cast<const words4 *>(b.k + at + d), y = *reinterpret_cast<const words4 *>(q + d);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            s = fmaf(E::load((uint16_t)(x[i / 2] >> (16 * (i % 2)))), E::load((uint16_t)(y[i / 2] >> (16 * (i % 2)))), s);
        }
      }
      const float top = fmaxf(m, wave_reduce<MaxF>(s));
      if (__any(s != s)) l = __builtin_nanf("");
      if (top == -__builtin_inff()) continue;
      const float factor = __builtin_amdgcn_exp2f((m - top) * a.c);
      m = top;
      const float w = key_weight(page >= 0, s, m, a.c);
      l = fmaf(l, factor, wave_reduce<SumF>(w));
      o = rescaled(o, factor);
      const uint64_t counts = __ballot(page >= 0 && s != -__builtin_inff());
      for (int j0 = 0; j0 < 64; j0 += 8) {
        words2 x[8];
        float wj[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          wj[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), j0 + j));
          const int64_t v = (int64_t)__builtin_amdgcn_readlane((int)(at >> 32), j0 + j) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)at, j0 + j);
          x[j] = words2{0, 0};
          if ((counts >> (j0 + j) & 1) && 4 * lane < b.dim) x[j] = *reinterpret_cast<const words2 *>(b.v + v + 4 * lane);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (counts >> (j0 + j) & 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = E::load((uint16_t)(x[j][i / 2] >> (16 * (i % 2))));
              o[i] = fmaf(fabsf(v) < __builtin_inff() ? wj[j] : 1.0f, v, o[i]);
            }
          }
      }
    }
    const Place place = place_of(a, r, head, row, part_of(parts, row - r.first), m, l, lane == 0);
    if (4 * lane < b.dim) place.put<E>(4 * lane, o);
  }
}

constexpr int kChunkKeys = 64;  // keys of a tile: a group of 16 to each of four waves

// What a workgroup of 128 x QB rows keeps in LDS: two buffers of a tile's keys and
// values.
template <int D>
struct ChunkTiles {
  static constexpr int KT = kChunkKeys, BYTES = KT * D * 2;
  int8_t tile[2][2][BYTES];
};

// 128 x QB rows, 32 x QB to each of four waves, over the key tiles [t0, t1), from
// t0 + turn on and round to it again; they come by two buffers, the next one loaded
// while one is worked on.
template <typename E, int D, int QB>
__device__ __forceinline__ void attend_rows(const AttentionArgs &a, const Rows &r, int head, int t0, int t1, int turn,
                                            int64_t parts, ChunkTiles<D> &lds, int lane, int wave) {
  constexpr int KT = kChunkKeys, GROUPS = KT / 16;
  typedef GroupLoads<D> Loads;
  const Paged &b = a.b;
  typedef WaveTile<E, D, QB, KT> Tile;
  Tile w;
  w.start(a, r, head, wave * 32 * QB, lane);

  uint32_t off_k[Loads::kLoads], off_v[Loads::kLoads];
  Loads::offsets(b, lane, false, off_k);
  Loads::offsets(b, lane, true, off_v);
  // lane i: the page of group i of the tile that is fetched next.  The number is looked
  // at a tile later than it is asked for (the asm keeps the compiler from looking at
  // once), since a wait for it is a wait for all loads before it.
  int pages;
  const int tiles = t1 - t0;
  const auto tile_at = [&](int n) { return t0 + n + turn < t1 ? t0 + n + turn : n + turn - tiles + t0; };
  const auto find_pages = [&](int n) {
    const int i = (tile_at(n) * KT + 16 * (lane % GROUPS)) >> b.page_shift;
    pages = -1;
    if (n < tiles && i < b.table_pages) pages = b.page_table[(int64_t)r.seq * b.table_ld + i];
  };
  const auto settle = [&]() {
    asm volatile("" : "+v"(pages));
    pages = (uint32_t)pages < (uint32_t)b.pages ? pages : -1;
  };
  const auto there_of = [&]() { return (uint32_t)__ballot(pages >= 0) & ((1u << GROUPS) - 1); };
  const auto fetch = [&](int n) {  // a wave fetches a group's keys and values
    const int key0 = tile_at(n) * KT + 16 * wave, page = __builtin_amdgcn_readlane(pages, wave);
    FB_LDS int8_t *const k = (FB_LDS int8_t *)lds.tile[n % 2][0] + wave * 16 * D * 2, *const v = (FB_LDS int8_t *)lds.tile[n % 2][1] + wave * 16 * D * 2;
    Loads::template load<false>(group_of(b, b.k, head, key0, page, r), lane, off_k, k);
    Loads::template load<false>(group_of(b, b.v, head, key0, page, r), lane, off_v, v);
  };
  find_pages(0);
  settle();
  uint32_t there = there_of();
  if (tiles > 0) fetch(0);
  find_pages(1);
  const int first_row = r.first + wave * 32 * QB, end_row = min(first_row + 32 * QB, r.count);
  for (int n = 0; n < tiles; ++n) {
    const int buf = n % 2, key0 = tile_at(n) * KT;
    wait_and_meet<0>();
    const uint32_t now = there;
    settle();
    there = there_of();
    if (n + 1 < tiles) fetch(n + 1);
    find_pages(n + 2);
    const bool border = key0 + KT - 1 > r.p_lo || (a.window && key0 <= r.p_hi - a.window);
    typename Tile::Scores s;
    typename Tile::Weights p;
    w.scores(lds.tile[buf][0], lane, s);
    w.mask(s, border || now != (1u << GROUPS) - 1 || key0 + KT > r.hi, key0, now, lane);
    __builtin_amdgcn_s_setprio(0);  // the other workgroup's products before this one's weights
    w.weights(a.c, s, p);
    w.add_values(lds.tile[buf][1], lane, p);
    __builtin_amdgcn_s_setprio(1);
  }
  if (w.unclean(a.c)) {
    rows_one_by_one<E>(a, r, head, parts, first_row, end_row, 1, t0 * KT, t1 * KT, lane);
    return;
  }
#pragma unroll
  for (int x = 0; x < QB; ++x) {
    const int row = first_row + 32 * x + lane % 32;
    const float l = other_half_sum(w.l[x]);
    if (row >= end_row) continue;
    const Place place = place_of(a, r, head, row, part_of(parts, row - r.first), w.m[x], l, lane < 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * i + 8 * j + 4 * (lane / 32);
        if (d < b.dim)
          place.put<E>(d, f32x4{w.o[i][x][4 * j], w.o[i][x][4 * j + 1], w.o[i][x][4 * j + 2], w.o[i][x][4 * j + 3]});
      }
  }
}

// Workgroups that a CU holds: with 256 dimensions the registers of a wave and the
// LDS are enough for one (two of 32-key tiles spill, and run at 690 TFLOP/s for 824).
template <int D>
constexpr int kChunksPerCu = D == 256 ? 1 : 2;

// One row tile and key head to a workgroup.
template <typename E, int D, int QB>
__global__ __launch_bounds__(256, kChunksPerCu<D>) void attention_chunk_kernel(const AttentionArgs a) {
  constexpr int KT = kChunkKeys;
  __shared__ __align__(1024) ChunkTiles<D> lds;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // key heads go to the XCDs in turn, so that the workgroups that share one's
  // keys share an L2; the last tiles, which see most, start first
  const int head = blockIdx.x % a.b.kv_heads, tile = a.tiles - 1 - blockIdx.x / a.b.kv_heads;
  const Rows r = rows_of<128 * QB>(a, tile, lane);
  if (r.count == 0) return;
  attend_rows<E, D, QB>(a, r, head, r.lo / KT, (r.hi + KT - 1) / KT, 0, -1, lds, lane, wave);
}

// Where there are few row tiles: the key tiles of all row tiles and heads, one behind
// the other, divided into equal shares, one to a workgroup.  A share is shorter than
// most row tiles' keys, so it is a run of one of them, or the end of one and the
// beginning of the next.  A workgroup has at most two parts for the join: number 2 g
// of a row tile that it goes on with and 2 g + 1 of one that it begins and does not
// end.
//
// The number of key tiles before each row tile; a row tile without keys counts as
// one, so that its rows are written.  A thread to a tile, kTilesMost of them.
constexpr int kTilesMost = 4096;
template <int BM>
__global__ __launch_bounds__(1024) void attention_count_kernel(const AttentionArgs a) {
  constexpr int KT = kChunkKeys;
  __shared__ int sums[16];
  const Paged &b = a.b;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int total = 0;
  for (int base = 0; base < a.tiles; base += 1024) {
    const int tile = base + (int)threadIdx.x;
    int n = 0;
    if (tile < a.tiles) {
      // the sequence: the last one whose tiles begin at or before this one
      int lo = 0, hi = b.seqs;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2, start = b.seq_starts ? max(0, min(b.seq_starts[mid], b.tokens)) : mid;
        if ((int)((int64_t)start * a.group / BM) + mid <= tile) lo = mid;
        else hi = mid - 1;
      }
      if (lo < b.seqs) {
        const int start = b.seq_starts ? b.seq_starts[lo] : lo, next = b.seq_starts ? b.seq_starts[lo + 1] : lo + 1;
        const Rows r = rows_at<BM>(a, tile, Found{lo, start, next, b.kv_lens[lo]});
        if (r.count) n = max(1, (r.hi + KT - 1) / KT - r.lo / KT);
      }
    }
    int sum = n;  // of the lanes up to this one
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    int ahead = total;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) ahead += sums[w];
      total += sums[w];
    }
    if (tile < a.tiles) a.before[tile] = ahead + sum - n;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.before[a.tiles] = total;
}

// Key tiles to a workgroup: equal shares, but none so small that its parts are most
// of its work.  (The host has seen to it that all key tiles are below 2^31.)
constexpr int kLeastShare = 8;
__device__ __forceinline__ int share_of(const AttentionArgs &a, int all) { return max(kLeastShare, (all + a.workgroups - 1) / a.workgroups); }

// The tile that has key tile `in` of a head: the last one that begins at or before
// it (tiles without rows, which take no room, begin with the next one).
__device__ __forceinline__ int tile_with(const AttentionArgs &a, int in, int lane) {
  int tile = 0, n = a.tiles - 1;
  while (n > 0) {
    const int step = (n + 63) / 64, j = (lane + 1) * step;
    const int c = __popcll(__ballot(j <= n && a.before[tile + j] <= in));
    tile += c * step;
    n = min(step - 1, n - c * step);
  }
  return tile;
}

template <typename E, int D, int QB>
__global__ __launch_bounds__(256, kChunksPerCu<D>) void attention_balanced_kernel(const AttentionArgs a) {
  constexpr int KT = kChunkKeys, BM = 128 * QB;
  __shared__ __align__(1024) ChunkTiles<D> lds;
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // an XCD's workgroups have consecutive shares: the same head's, mostly
  const int g = blockIdx.x % 8 * (a.workgroups / 8) + blockIdx.x / 8;
  const int per_head = a.before[a.tiles], all = per_head * a.b.kv_heads, share = share_of(a, all);
  const int first = (int)min((int64_t)g * share, (int64_t)all);
  // Workgroups that share a head's keys should read the same ones at about the same
  // time, so that one of them finds what another has loaded in the L2: a share's key
  // tiles are taken in the order of their number modulo the share's length.  So the
  // beginning of the next row tile goes before the end of the last one, and a run
  // starts at the multiple of the length that lies in it.
  int end = (int)min((int64_t)first + share, (int64_t)all);
#pragma unroll 1
  while (end > first) {
    const int head = (end - 1) / per_head, in = (end - 1) % per_head;
    const int tile = tile_with(a, in, lane), before = a.before[tile], size = a.before[tile + 1] - before;
    const int to = in + 1 - before, from = max(0, to - (end - first));
    const Rows r = rows_of<BM>(a, tile, lane);
    const int begin = r.lo / KT, last = (r.hi + KT - 1) / KT, whole = (from + share - 1) / share * share;
    __syncthreads();  // the tiles of the last rows have been read
    attend_rows<E, D, QB>(a, r, head, begin + from, min(begin + to, last), whole < min(to, last - begin) ? whole - from : 0,
                          from == 0 && to == size ? -1 : ((int64_t)2 * g + (from == 0)) * BM, lds, lane, wave);
    end -= to - from;
  }
}

// The parts of the row tiles that several workgroups had, joined.  A wave has two
// rows, or two pairs of them where half its lanes hold a row, and loads four parts of
// each at once (a row to a wave takes 22 us instead of 13 for 4136 rows of 8 heads:
// each wave looks its tile up before it loads).
constexpr int kGatherRows = 2;
template <typename E, int BM>
__global__ __launch_bounds__(256) void attention_gather_kernel(const AttentionArgs a) {
  const Paged &b = a.b;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, pair = b.dim <= 128 ? 2 : 1;
  const int per_head = a.before[a.tiles], share = share_of(a, per_head * b.kv_heads);
  const int blocks = BM / (4 * kGatherRows * pair), rest = blockIdx.x / blocks, head = rest % b.kv_heads, tile = rest / b.kv_heads;
  const int n = a.before[tile + 1] - a.before[tile];
  if (n == 0) return;
  const int at = head * per_head + a.before[tile], g0 = at / share, g1 = (at + n - 1) / share;
  if (g0 == g1) return;
  const Rows r = rows_of<BM>(a, tile, lane);
  const int d = 4 * (lane % (64 / pair)), rows = min(BM, r.count - r.first);
  const int first = ((int)(blockIdx.x % blocks) * 4 + wave) * kGatherRows * pair + lane / (64 / pair);
  float m[kGatherRows], sum[kGatherRows];
  f32x4 o[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    m[i] = -__builtin_inff();
    sum[i] = 0.0f;
    o[i] = f32x4{0, 0, 0, 0};
  }
#pragma unroll 4
  for (int g = g0; g <= g1; ++g) {
    // the first workgroup began the tile, whether or not its share begins with it
    const int64_t from = ((int64_t)2 * g + (g == g0)) * BM;
    float now_m[kGatherRows], l[kGatherRows];
    f32x4 v[kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      const int64_t p = from + min(first + i * pair, rows - 1);
      now_m[i] = a.stats[2 * p];
      l[i] = a.stats[2 * p + 1];
      v[i] = f32x4{0, 0, 0, 0};
      if (d < b.dim) v[i] = *reinterpret_cast<const f32x4 *>(a.part + p * b.dim + d);
    }
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      const float top = fmaxf(m[i], now_m[i]);
      const float old = m[i] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m[i] - top) * a.c);
      const float now = now_m[i] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((now_m[i] - top) * a.c);
      m[i] = top;
      sum[i] = fmaf(sum[i], old, l[i] * now);
      o[i] = rescaled(o[i], old) + rescaled(v[i], now);
    }
  }
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    if (first + i * pair >= rows) continue;
    const Place place = place_of(a, r, head, r.first + first + i * pair, -1, m[i], sum[i], d == 0);
    if (d < b.dim) place.put<E>(d, o[i]);
  }
}

// Up to 32 rows: the waves share them and split the keys, each with a place of its
// own for a tile's keys and one for its values, loaded again as soon as they have
// been read, so that nothing waits for another wave before the end and a wave
// always has loads in flight.  Keys and values are marked as read once (64
// sequences of up to 8192 keys: 163 us for 181), which they are where a sequence has one
// row tile; where it has several (a chunk among single tokens, more than 32 query
// heads to a key head) each of them asks for them.  Eight waves of 16 KiB: a wave's chain of products and
// weights is long for a single query, and two to a SIMD hide it better than more
// tiles ahead of fewer waves.
template <int D>
struct Few {
  static constexpr int W = D == 256 ? 4 : 8, KT = 32, BYTES = KT * D * 2;
};
template <typename E, int D>
__global__ __launch_bounds__(64 * Few<D>::W) void attention_few_kernel(const AttentionArgs a) {
  typedef Few<D> F;
  constexpr int W = F::W, KT = F::KT, BYTES = F::BYTES;
  typedef GroupLoads<D> Loads;
  typedef WaveTile<E, D, 1, KT> Tile;
  __shared__ __align__(1024) int8_t lds[W * 2 * BYTES];  // the waves' sums, 32 x D floats each, take it over
  __shared__ float stats[2][W][32];
  __shared__ bool any_bad[W];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Paged &b = a.b;
  const int head = blockIdx.x % b.kv_heads, rest = blockIdx.x / b.kv_heads;
  const int split = rest % a.splits, tile = rest / a.splits;
  const Rows r = rows_of<32>(a, tile, lane);
  if (r.count == 0) return;

  const int begin = r.lo / KT, all = max(0, (r.hi + KT - 1) / KT - begin), per = (all + a.splits - 1) / a.splits;
  const int t0 = begin + min(split * per, all), t1 = begin + min((split + 1) * per, all);
  const int64_t parts = a.splits > 1 ? (((int64_t)tile * b.kv_heads + head) * a.splits + split) * 32 : -1;
  Tile w;
  w.start(a, r, head, 0, lane);

  uint32_t off_k[Loads::kLoads], off_v[Loads::kLoads];
  Loads::offsets(b, lane, false, off_k);
  Loads::offsets(b, lane, true, off_v);
  int8_t *const kt = lds + wave * 2 * BYTES, *const vt = kt + BYTES;
  // lane 2 i + g of `pages`: the page of the group g of the wave's tile number i
  // after the last look-up, made every 32 tiles
  int pages = -1;
  const auto page = [&](int n, int g) { return __builtin_amdgcn_readlane(pages, n % 32 * 2 + g); };
  // The wave's tile number n.  Loads of tiles that do not exist read an empty
  // buffer, so that every tile counts the same number of loads.
  const auto fetch = [&](int n, const uint16_t *cache, const uint32_t (&off)[Loads::kLoads], int8_t *dst) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
      Loads::template load<true>(group_of(b, cache, head, (t0 + wave + n * W) * KT + 16 * g, page(n, g), r), lane, off, (FB_LDS int8_t *)dst + g * 16 * D * 2);
  };
  const auto find_pages = [&](int n) {
    if (n % 32 == 0) {
      const int t = t0 + wave + (n + lane / 2) * W;
      pages = t < t1 ? page_of(b, r.seq, t * KT + 16 * (lane % 2)) : -1;
    }
  };
  find_pages(0);
  fetch(0, b.k, off_k, kt);
  fetch(0, b.v, off_v, vt);
#pragma unroll 1
  for (int n = 0; t0 + wave + n * W < t1; ++n) {
    const int key0 = (t0 + wave + n * W) * KT;
    const bool border = key0 + KT - 1 > r.p_lo || (a.window && key0 <= r.p_hi - a.window);
    const uint32_t there = (page(n, 0) >= 0) | (page(n, 1) >= 0) << 1;
    typename Tile::Scores s;
    typename Tile::Weights p, rest;
    find_pages(n + 1);
    wait_for_loads<2 * Loads::kLoads>();
    w.scores(kt, lane, s);
    wait_for_reads();
    fetch(n + 1, b.k, off_k, kt);
    w.mask(s, border || there != 3 || key0 + KT > r.hi, key0, there, lane);
    w.exact_weights(a.c, s, p, rest);
    wait_for_loads<2 * Loads::kLoads>();
    w.add_values(vt, lane, p, &rest);
    wait_for_reads();
    fetch(n + 1, b.v, off_v, vt);
  }

  // Join the waves.
  const float l = other_half_sum(w.l[0]);
  wait_and_meet<0>();
  if (lane < 32) {
    stats[0][wave][lane] = w.m[0];
    stats[1][wave][lane] = l;
  }
  bool bad = w.unclean(a.c);
  if (lane == 0) any_bad[wave] = bad;
  __syncthreads();
  const int rows = min(32, r.count - r.first);
#pragma unroll
  for (int v = 0; v < W; ++v) bad = bad || any_bad[v];
  if (bad) {
    rows_one_by_one<E>(a, r, head, parts, r.first + wave, r.first + rows, W, t0 * KT, t1 * KT, lane);
    return;
  }
  const int mine_row = lane % 32;
  float top = -__builtin_inff();
#pragma unroll
  for (int v = 0; v < W; ++v) top = fmaxf(top, stats[0][v][mine_row]);
  const float factor = w.m[0] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((w.m[0] - top) * a.c);
  // four floats to a place, places exchanged by the row so that rows fall into
  // different banks
  float *sums = reinterpret_cast<float *>(lds);
  const auto sum_at = [](int row, int place) { return (place ^ row % 16) * 4; };
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4 *>(sums + (wave * 32 + mine_row) * D + sum_at(mine_row, 8 * i + 2 * j + lane / 32)) =
          f32x4{w.o[i][0][4 * j], w.o[i][0][4 * j + 1], w.o[i][0][4 * j + 2], w.o[i][0][4 * j + 3]} * factor;
  __syncthreads();
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
      o += *reinterpret_cast<const f32x4 *>(sums + (v * 32 + row) * D + sum_at(row, d / 4));
    }
    place_of(a, r, head, r.first + row, part_of(parts, row), big, sum, d == 0).put<E>(d, o);
  }
}

// The splits' parts of a tile's 32 rows joined, eight rows to a wave.
template <typename E>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttentionArgs a) {
  const int lane = threadIdx.x % 64, head = blockIdx.x % a.b.kv_heads, tile = blockIdx.x / a.b.kv_heads;
  const Rows r = rows_of<32>(a, tile, lane);
  if (r.count == 0) return;
  for (int x = threadIdx.x / 64; x < min(32, r.count - r.first); x += 4) {
    const int64_t first = (int64_t)blockIdx.x * a.splits * 32 + x;
    float m = -__builtin_inff(), l = 0.0f;
    if (lane < a.splits) {
      m = a.stats[2 * (first + lane * 32)];
      l = a.stats[2 * (first + lane * 32) + 1];
    }
    const float top = wave_reduce<MaxF>(m);
    const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.c);
    const float sum = wave_reduce<SumF>(f * l);  // a split without keys has l = 0; one whose l is NaN counts whatever its m
    const float *part = a.part + first * a.b.dim + 4 * lane;
    // eight splits' parts are in flight; those of splits without keys hold zeros
    const auto joined = [&](auto scaled) {
      f32x4 o{0, 0, 0, 0};
      for (int base = 0; base < a.splits; base += 8) {
        f32x4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = f32x4{0, 0, 0, 0};
          if (base + i < a.splits && 4 * lane < a.b.dim) v[i] = *reinterpret_cast<const f32x4 *>(part + (int64_t)(base + i) * 32 * a.b.dim);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float fs = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), (base + i) % 64));
          if (base + i < a.splits) o += scaled(v[i], fs);
        }
      }
      return o;
    };
    f32x4 o = joined([](f32x4 v, float fs) { return v * fs; });
    const f32x4 z = o * 0.0f;
    if (__any(!(z[0] + z[1] + z[2] + z[3] == 0.0f))) o = joined(rescaled);  // rare, and 0.3 us for all rows
    const Place place = place_of(a, r, head, r.first + x, -1, top, sum, lane == 0);
    if (4 * lane < a.b.dim) place.put<E>(4 * lane, o);
  }
}

}  // namespace fluxbin
