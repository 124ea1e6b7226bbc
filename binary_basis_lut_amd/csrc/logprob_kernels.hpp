// logprob_kernels.hpp -- log probabilities of given tokens, the entropy and the
// best alternatives of every row of logits, in one pass over the row.
//
// Mathematics.  With z_j = s x_j (s > 0 the logit scale), c = s log2(e) and m
// the largest x_j:
//     d_j = c (x_j - m),  S = sum 2^d_j,  D = sum 2^d_j d_j
//     log p_j = s (x_j - m) - ln2 log2 S,  entropy = ln2 (log2 S - D / S).
// A thread keeps (m, S, D) for the elements it has seen; two such triples are
// joined by moving both to the larger m: with e = c (m_old - m_new) (<= 0),
// S -> 2^e S and D -> 2^e (D + e S).  All of it is fp32.  The difference is
// taken before the product, so that rows at the type's lowest value (a common
// mask) stay finite; 2^d d is taken with d held at -200 or above, where 2^d is
// 0, so that a masked logit (-inf) adds 0 and not NaN; NaN and +inf logits make
// S NaN.
//
// Alternatives are ordered by key: the logit's bits as an ordered integer above
// the complement of its index, so of equal logits the lower index is first.
#pragma once

#include "elements.hpp"
#include "wave_ops.hpp"

namespace fluxbin {

struct LogprobArgs {
  const void *logits;
  const int64_t *targets;                // null: no targets
  float *logprob, *entropy, *top_logprob;  // entropy may be null
  int64_t *top_index;
  uint8_t *workspace;                    // splits > 1: the partial results
  int64_t rows, ld;
  int32_t vocab, top_k, splits, split_len;  // split_len: columns per split, a multiple of 64
  float scale;
};

// A workgroup of T threads takes a slice of T x kLpUnits units of eight columns at
// a time: 1024 threads where few rows, each within one slice, have to fill the
// chip (such a row needs no join of splits), else 256; rows of a few hundred
// columns go to one wave each.
constexpr int kLpFew = 1024, kLpMany = 256, kLpTiny = 64;
constexpr int kLpUnits = 4;                  // units of eight per thread and slice
constexpr int kLpSmall = kLpMany * kUnit;    // splits up to this length go by single columns
constexpr int kLpTinyCols = kLpTiny * kUnit;  // rows up to this length, by single columns too
constexpr int kLpFewCols = kLpFew * kUnit * kLpUnits;  // columns that kLpFew threads hold in registers
constexpr int kLpMaxTop = 64;
static_assert(kLpUnits * kUnit == 32, "a thread marks its elements of a slice in one word");
constexpr int kLpCap = 512;                  // candidate keys that LDS holds
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

// The next value above f (NaN above infinity: no value is as large).
__device__ __forceinline__ float above(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 counts as +0
  return __builtin_bit_cast(float, (b >> 31) ? b - 1 : b + 1);
}

struct Stats {
  float m, s, d;  // largest x, sum of 2^(c (x - ref(m))), that sum weighted with its exponents
};

// The reference of a largest value; 0 where there is none yet.
__device__ __forceinline__ float ref(float m) { return m == kNegInf ? 0.0f : m; }

__device__ __forceinline__ Stats join(Stats a, Stats b, float c) {
  Stats r;
  r.m = fmaxf(a.m, b.m);
  const float ea = fmaxf((ref(a.m) - ref(r.m)) * c, -200.0f), eb = fmaxf((ref(b.m) - ref(r.m)) * c, -200.0f);
  // a side without a finite logit has s = d = 0 (or NaN): its shift is of no account
  const float ta = a.m == kNegInf ? 0.0f : ea, tb = b.m == kNegInf ? 0.0f : eb;
  const float fa = __builtin_amdgcn_exp2f(ta), fb = __builtin_amdgcn_exp2f(tb);
  r.s = a.s * fa + b.s * fb;
  r.d = fmaf(ta, a.s, a.d) * fa + fmaf(tb, b.s, b.d) * fb;
  return r;
}

// Ordered key of element `index` with value x; 0 is below every key.
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  const int b = __builtin_bit_cast(int, x + 0.0f);  // -0 ranks as +0
  const uint32_t o = (uint32_t)b ^ (b < 0 ? 0xffffffffu : 0x80000000u);
  return (uint64_t)o << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, (o >> 31) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int index_of(uint64_t key) { return (int)~(uint32_t)key; }

// The joined statistics of a wave, in every lane: the largest x first, so that
// each lane moves its own sums once.
__device__ __forceinline__ Stats join_wave(Stats a, float c) {
  Stats r;
  r.m = wave_reduce<MaxF>(a.m);
  const float t = a.m == kNegInf ? 0.0f : fmaxf((a.m - ref(r.m)) * c, -200.0f), f = __builtin_amdgcn_exp2f(t);
  r.s = wave_reduce<SumF>(a.s * f);
  r.d = wave_reduce<SumF>(fmaf(t, a.s, a.d) * f);
  return r;
}

// What the waves of a workgroup share while they pick the best keys.
template <int T>
struct LpShared {
  uint64_t cand[kLpCap];
  uint64_t list[kLpMaxTop];  // the best keys, in order; 0 past their count
  Stats wave[T / 64];
  uint64_t wkey[T / 64];
  float wthr[T / 64];
  int count;
};

// cand[0, n) -> the best top_k of them in list, in order.
template <int T>
__device__ __forceinline__ void select_by_rank(LpShared<T> &sh, int n, int top_k) {
  if (threadIdx.x < (unsigned)kLpMaxTop) sh.list[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += T) {
    const uint64_t k = sh.cand[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += sh.cand[j] > k;
    if (rank < top_k) sh.list[rank] = k;
  }
  __syncthreads();
}

template <int T>
__device__ __forceinline__ uint64_t block_max_key(LpShared<T> &sh, uint64_t k) {
  k = wave_reduce<MaxKey>(k);
  __syncthreads();
  if (threadIdx.x % 64 == 0) sh.wkey[threadIdx.x / 64] = k;
  __syncthreads();
  k = sh.wkey[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) k = sh.wkey[i] > k ? sh.wkey[i] : k;
  return k;
}

// The n-th largest (n >= 1) of the wave's values, -inf where fewer are above it.
__device__ __forceinline__ float wave_nth(float v, int n) {
  if (n > 4) {  // by the number of larger values, 64 independent comparisons
    int larger = 0;
#pragma unroll
    for (int j = 0; j < 64; ++j)
      larger += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), j)) > v;
    return -wave_reduce<MaxF>(larger < n ? -v : kNegInf);  // the least of those with fewer than n above them
  }
  float m = wave_reduce<MaxF>(v);
  while (--n > 0) {
    const uint64_t at = __ballot(v == m);
    if (v == m && (threadIdx.x % 64) == (unsigned)__builtin_ctzll(at)) v = kNegInf;
    m = wave_reduce<MaxF>(v);
  }
  return m;
}

// The joined statistics of a workgroup, in every thread.
template <int T>
__device__ __forceinline__ Stats join_block(LpShared<T> &sh, Stats st, float c) {
  st = join_wave(st, c);
  if (threadIdx.x % 64 == 0) sh.wave[threadIdx.x / 64] = st;
  __syncthreads();
  if (T == 64) return st;
  const unsigned lane = threadIdx.x % 64;
  return join_wave(lane < T / 64 ? sh.wave[lane] : Stats{kNegInf, 0.0f, 0.0f}, c);
}

// A row's target and its logit, fetched by thread 0 ahead of their use (first
// the index, with a row's other loads behind it, then the logit).
struct Target {
  int64_t index;
  float x;
};

__device__ __forceinline__ Target target_index(const LogprobArgs &a, int64_t row) {
  return Target{a.targets && threadIdx.x == 0 ? a.targets[row] : -1, 0.0f};
}
template <typename E>
__device__ __forceinline__ void target_logit(const LogprobArgs &a, int64_t row, Target &t) {
  if (t.index >= 0 && t.index < a.vocab) t.x = E::load(((const typename E::raw *)a.logits)[row * a.ld + t.index]);
}

// Writes a row's results from its joined statistics and its ordered keys.
__device__ __forceinline__ void write_row(const LogprobArgs &a, int64_t row, Stats st, const uint64_t *list, Target target) {
  const float m = ref(st.m);
  const float l2 = __builtin_amdgcn_logf(st.s);  // S = 0 (nothing left): -inf
  const bool none = st.s == 0.0f;
  auto lp = [&](float x) { return none ? kNegInf : (x - m) * a.scale - kLn2 * l2; };
  const int t = threadIdx.x;
  if (t == 0) {
    if (a.targets) {
      float v = 0.0f;  // a negative target is no target
      if (target.index >= a.vocab) v = __builtin_nanf("");
      else if (target.index >= 0) v = lp(target.x);
      a.logprob[row] = v;
    }
    if (a.entropy) a.entropy[row] = none ? 0.0f : kLn2 * (l2 - st.d / st.s);
  }
  if (t < a.top_k) {
    const uint64_t k = list[t];
    a.top_logprob[row * a.top_k + t] = k ? lp(value_of(k)) : __builtin_nanf("");
    a.top_index[row * a.top_k + t] = k ? index_of(k) : -1;
  }
}

// Bytes of one split's partial result: the statistics, then top_k keys.
__host__ __device__ inline int64_t lp_part_bytes(int top_k) { return 16 + 8 * (int64_t)top_k; }

// One workgroup: one split of one row.  splits == 1 writes the row's results,
// else the split's partial result goes to the workspace.
//
// Alternatives without sorting: the first slice gives a lower bound of the
// top_k-th value (each wave's ceil(top_k / waves)-th largest thread maximum,
// the least of them: at least top_k elements reach it), and only elements above
// the bound become candidates in LDS.  After 2, 4, 8, ... slices the candidates
// are reduced to the best top_k and the bound rises to the last of them, so
// their number stays near top_k (1 + ln 2) however long the row is.  Equal
// elements of later slices have higher indices and lose, hence "above".  Rows
// that defeat this (long runs of equal logits, ascending rows, fewer than top_k
// logits left unmasked) are taken again, one key at a time.
//
// SMALL (splits of at most kLpSmall columns): a thread takes single columns, T
// apart, instead of eight in a row, so that all threads have their part of a
// short row and its bound is close.
//
// Bound by the HBM read for fp32 rows (4096 x 32000, 524 MB, in 92 us = 5.7 TB/s);
// for 16-bit rows the exponential, a quarter-rate instruction, and the
// conversions weigh as much (about 11 issue slots per element; 4096 x 32000
// fp16 in 68 us = 3.9 TB/s).  Few rows are latency: 6 us per kernel at 2000 to
// 5000 columns, 9 at 32000, or 6 and 4 more for the join where a row is split.
template <typename E, bool SMALL, int T>
__global__ __launch_bounds__(T) void logprob_rows_kernel(const LogprobArgs a) {
  typedef typename E::raw raw;
  constexpr int kWaves = T / 64, U = SMALL ? 1 : kLpUnits, kStep = T * kUnit, kSlice = kStep * U;
  __shared__ LpShared<T> sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x % a.splits);
  const int begin = split * a.split_len, end = min(a.vocab, begin + a.split_len);
  const raw *x = (const raw *)a.logits + row * a.ld;
  const float c = a.scale * kLog2e;
  Stats st{kNegInf, 0.0f, 0.0f};
  float thr = kNegInf, least = kNegInf;  // candidates are >= least
  int slice = 0;
  bool full = false;  // more candidates than LDS holds
  if (tid == 0) sh.count = 0;
  Target target = a.splits == 1 ? target_index(a, row) : Target{-1, 0.0f};
  for (int at0 = begin; at0 < end; at0 += kSlice, ++slice) {
    typename E::unit v[U];
    const int units = min(U, (end - at0 + kStep - 1) / kStep);  // units that hold columns
    float tm = kNegInf;
    if (SMALL) {
      v[0].fill(E::round(kNegInf));
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (at0 + i * T + tid < end) v[0].put(i, x[at0 + i * T + tid]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = load_part<E, false, int>(x, at0 + (u * T + tid) * kUnit, end, kNegInf);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= units) break;
      if (!SMALL) settle_part<E, false, int>(v[u], at0 + (u * T + tid) * kUnit, end, kNegInf);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) tm = fmaxf(tm, v[u].get(i));
    }
    {
      const float m = fmaxf(st.m, tm), M = ref(m);
      Stats now{m, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= units) break;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          const float d = (v[u].get(i) - M) * c, e = __builtin_amdgcn_exp2f(d);
          now.s += e;
          now.d = fmaf(e, fmaxf(d, -200.0f), now.d);
        }
      }
      st = join(st, now, c);
    }
    if (a.top_k == 0) continue;
    if (slice == 0) {
      // of the waves that hold columns in every lane, or of the first
      const int waves = max(1, min(kWaves, (end - begin) / (64 * (SMALL ? 1 : kUnit))));
      const float w = wave_nth(tm, (a.top_k + waves - 1) / waves);
      if (tid % 64 == 0) sh.wthr[tid / 64] = w;
      __syncthreads();
      thr = sh.wthr[0];
      for (int i = 1; i < waves; ++i) thr = fminf(thr, sh.wthr[i]);
      least = fmaxf(thr, -3.402823466e38f);
    }
    if (!full && tm >= least) {
      uint32_t mask = 0;  // element j of the slice's 8 U at bit 8 U - 1 - j
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) mask = mask + mask + (v[u].get(i) >= least ? 1u : 0u);
      int p = atomicAdd(&sh.count, (int)__builtin_popcount(mask));
      while (mask) {  // few
        const int j = __builtin_clz(mask) - (32 - kUnit * U);
        const int at = at0 + (SMALL ? j * T + tid : ((j / kUnit) * T + tid) * kUnit + j % kUnit);
        mask &= ~(1u << (kUnit * U - 1 - j));
        if (p < kLpCap) sh.cand[p] = key_of(E::unit::pick(v, j), at);
        ++p;
      }
    }
    if (slice == 0) least = above(thr);
    if (slice > 0 && (slice & (slice + 1)) == 0 && at0 + kSlice < end && !full) {
      __syncthreads();
      const int n = sh.count;
      full = n > kLpCap;
      if (!full && n >= a.top_k) {
        select_by_rank(sh, n, a.top_k);
        if (tid < a.top_k) sh.cand[tid] = sh.list[tid];
        if (tid == 0) sh.count = a.top_k;
        least = above(value_of(sh.list[a.top_k - 1]));
      }
      __syncthreads();
    }
  }
  target_logit<E>(a, row, target);
  st = join_block(sh, st, c);  // its barrier stands behind the last candidates, too
  if (a.top_k > 0) {
    const int n = sh.count;
    if (!full && n >= a.top_k && n <= kLpCap) {
      select_by_rank(sh, n, a.top_k);
    } else {
      // the largest key below the last one, top_k times
      uint64_t below = ~0ull;
      for (int j = 0; j < a.top_k; ++j) {
        uint64_t best = 0;
        for (int at = begin + tid; at < end; at += T) {
          const float f = E::load(x[at]);
          const uint64_t k = key_of(f, at);
          if (f == f && k < below && k > best) best = k;
        }
        below = block_max_key(sh, best);
        if (tid == 0) sh.list[j] = below;
      }
      __syncthreads();
    }
  }
  if (a.splits == 1) {
    write_row(a, row, st, sh.list, target);
  } else {
    uint8_t *p = a.workspace + (row * a.splits + split) * lp_part_bytes(a.top_k);
    if (tid == 0) {
      float *f = (float *)p;
      f[0] = st.m;
      f[1] = st.s;
      f[2] = st.d;
    }
    if (tid < a.top_k) ((uint64_t *)(p + 16))[tid] = sh.list[tid];
  }
}

// Joins the splits of a row (at most kLpMany of them).
template <typename E>
__global__ __launch_bounds__(kLpMany) void logprob_join_kernel(const LogprobArgs a) {
  __shared__ LpShared<kLpMany> sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x, pb = lp_part_bytes(a.top_k);
  const uint8_t *base = a.workspace + row * a.splits * pb;
  const float c = a.scale * kLog2e;
  Target target = target_index(a, row);
  Stats st{kNegInf, 0.0f, 0.0f};
  // A lower bound of the row's top_k-th key: with t = ceil(top_k / splits), the
  // ceil(top_k / t)-th largest of the splits' t-th keys (each has t keys from it on).
  uint64_t mine = 0;
  const int t = a.top_k > 0 ? (a.top_k + a.splits - 1) / a.splits : 1;
  const uint64_t *list = (const uint64_t *)(base + (tid < a.splits ? tid : 0) * pb + 16);
  if (tid < a.splits) {
    const float *f = (const float *)(base + tid * pb);
    st = Stats{f[0], f[1], f[2]};
    if (a.top_k > 0) mine = list[t - 1];
    sh.cand[tid] = mine;
  }
  if (tid == 0) sh.count = 0;
  target_logit<E>(a, row, target);
  st = join_block(sh, st, c);
  if (a.top_k > 0) {
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < a.splits; ++i) rank += sh.cand[i] > mine || (sh.cand[i] == mine && i < tid);
    if (tid < a.splits && rank == (a.top_k + t - 1) / t - 1) sh.wkey[0] = mine;
    __syncthreads();
    const uint64_t bound = sh.wkey[0];
    for (int i = tid; i < a.splits * a.top_k; i += kLpMany) {
      const uint64_t k = ((const uint64_t *)(base + (i / a.top_k) * pb + 16))[i % a.top_k];
      if (k >= bound && k > 0) {
        const int p = atomicAdd(&sh.count, 1);
        if (p < kLpCap) sh.cand[p] = k;
      }
    }
    __syncthreads();
    const int n = sh.count;
    if (n <= kLpCap) {
      select_by_rank(sh, n, a.top_k);
    } else {
      // each split's list is in order: the largest head, top_k times
      int head = 0;
      for (int j = 0; j < a.top_k; ++j) {
        const uint64_t k = tid < a.splits && head < a.top_k ? list[head] : 0;
        const uint64_t best = block_max_key(sh, k);
        if (k == best && k) ++head;
        if (tid == 0) sh.list[j] = best;
      }
      __syncthreads();
    }
  }
  write_row(a, row, st, sh.list, target);
}

}  // namespace fluxbin
