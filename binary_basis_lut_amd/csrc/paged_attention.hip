// paged_attention.hip -- fluxbin_paged_attention: argument checks, the choice of a
// kernel and of the split of the keys, the launches.
#include <algorithm>

#include "attention_kernels.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kMaxGrid = ((int64_t)1 << 23) - 1;  // of 512 threads, HIP takes fewer than 2^32

// Sequences whose new tokens fill at most 32 rows of a key head on average go to
// the kernel whose waves share the rows and split the keys.  Where such tiles are
// fewer than fill the chip, the keys are split over workgroups too.
constexpr int64_t kFewRows = 32;
constexpr int64_t kMinKeys = 512;   // of a split
constexpr int64_t kMaxSplits = 64;  // the join's lanes

constexpr int64_t kChunkRows = 128;

// Whether equal shares of the key tiles are faster than a workgroup to a row tile
// and head: `units` key tiles that every row tile has, `busy` of these, in the times
// of a key tile measured with one workgroup to a CU (alone) and with all that it holds
// (full).  Between, some CUs hold one and some two, and the last of these ends the
// launch: 1.7 us to a key tile of 128 dimensions at 264 workgroups, 1.9 at 448, 2.1 at
// 504, for which 0.8 of the full time stands.  Counting the shares and joining their
// parts takes about kJoin.  With 128 dimensions and 64 heads to 8, us by shares and
// without (* the choice): 100 new tokens over 30000 93* and 590; 528 over 31000 611*
// and 813, over 8000 179* and 208, over 2000 75 and 68*; 640 over 31000 709* and 809,
// over 8000 214* and 221; 768 over 31000 838* and 855, over 8000 252 and 238*; 256 over
// 2000 49* and 50; 512 over 4000 109 and 95*.  From 512 workgroups on there are no
// shares, whatever the last round of workgroups leaves idle (1008 over 31000 1014, 1040,
// of 520 workgroups, 1588).  Without cached tokens the first row tiles are short and a
// share has many (2000 new tokens 122 and 58): only cached ones count.
constexpr double kJoin = 25.0;  // us
bool shares_pay(double units, int64_t busy, int64_t shares, int64_t dim) {
  const double alone = dim <= 64 ? 0.8 : dim <= 128 ? 1.4 : 2.6, full = dim <= 64 ? 1.4 : dim <= 128 ? 2.5 : 2.6;
  return units * (busy <= 256 ? alone : 0.8 * full) > units * full * (double)busy / (double)shares + kJoin;
}

struct Plan {
  bool few, balanced;
  int32_t splits, shares;
  int64_t tiles, parts;  // parts: rows of the workspace
};

// Of a batch with tokens and sequences.
Plan plan_of(const fluxbin_paged_batch &b, int64_t window) {
  const int64_t group = b.heads / b.kv_heads, per_seq = cdiv(b.tokens * group, b.seqs);
  const int64_t cap = b.table_pages * b.page_size, most = b.max_kv_len ? std::min(b.max_kv_len, cap) : cap;
  const int64_t keys = window ? std::min(most, window + b.tokens) : most;
  Plan p{};
  p.few = per_seq <= kFewRows;
  p.splits = 1;
  const int64_t rows = p.few ? kFewRows : kChunkRows;
  p.tiles = b.tokens * group / rows + b.seqs;
  const int64_t busy = std::max<int64_t>(1, b.seqs * cdiv(per_seq, rows) * b.kv_heads);
  if (p.few) {
    const int64_t room = b.dim <= 64 ? 512 : 256;  // workgroups that the chip's LDS holds
    p.splits = (int32_t)std::max<int64_t>(1, std::min({room / busy, cdiv(keys, kMinKeys), kMaxSplits}));
    p.parts = p.splits > 1 ? p.tiles * b.kv_heads * p.splits * kFewRows : 0;
  } else {
    p.shares = b.dim <= 128 ? 256 * kChunksPerCu<128> : 256 * kChunksPerCu<256>;
    p.balanced = busy < p.shares && p.tiles <= kTilesMost && p.tiles * b.kv_heads * cdiv(cap, 32) < (int64_t)1 << 30 &&
                 shares_pay((double)(keys - cdiv(b.tokens, b.seqs)) / kChunkKeys, busy, p.shares, b.dim);
    p.parts = p.balanced ? 2 * p.shares * kChunkRows : 0;
  }
  return p;
}

// Workgroups that join the parts of one row tile and head.
int64_t gather_blocks(int64_t dim) { return kChunkRows / (4 * kGatherRows * (dim <= 128 ? 2 : 1)); }

size_t before_bytes(const Plan &p) { return p.balanced ? (size_t)cdiv((p.tiles + 1) * 4, 256) * 256 : 0; }
size_t ws_bytes(const fluxbin_paged_batch &b, const Plan &p) { return before_bytes(p) + (size_t)(p.parts * (b.dim + 2)) * 4; }

template <typename E, int D>
void launch(const AttentionArgs &a, const Plan &p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.splits * a.b.kv_heads));
  if (p.few) {
    hipLaunchKernelGGL((attention_few_kernel<E, D>), grid, dim3(64 * Few<D>::W), 0, st, a);
    if (p.splits > 1) hipLaunchKernelGGL(attention_join_kernel<E>, dim3((unsigned)(p.tiles * a.b.kv_heads)), dim3(256), 0, st, a);
  } else if (p.balanced) {
    hipLaunchKernelGGL((attention_count_kernel<kChunkRows>), dim3(1), dim3(1024), 0, st, a);
    hipLaunchKernelGGL((attention_balanced_kernel<E, D, 1>), dim3(p.shares), dim3(256), 0, st, a);
    hipLaunchKernelGGL((attention_gather_kernel<E, kChunkRows>), dim3((unsigned)(p.tiles * a.b.kv_heads * gather_blocks(a.b.dim))), dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((attention_chunk_kernel<E, D, 1>), grid, dim3(256), 0, st, a);
  }
}

template <typename E>
void run(const AttentionArgs &a, const Plan &p, hipStream_t st) {
  if (a.b.dim <= 64) launch<E, 64>(a, p, st);
  else if (a.b.dim <= 128) launch<E, 128>(a, p, st);
  else launch<E, 256>(a, p, st);
}

}  // namespace

extern "C" {

fluxbin_status fluxbin_paged_attention_workspace_size(const fluxbin_paged_batch *batch, size_t *bytes) {
  const fluxbin_status st = check_paged(batch);
  if (st) return st;
  if (!bytes) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "bytes is NULL");
  // a window never takes more than none
  *bytes = batch->tokens && batch->seqs ? ws_bytes(*batch, plan_of(*batch, 0)) : 0;
  return ok();
}

fluxbin_status fluxbin_paged_attention(const fluxbin_paged_batch *batch, const void *q, int64_t ldq, float scale, int32_t window,
                                       void *out, int64_t ldo, float *lse, void *workspace, size_t workspace_bytes,
                                       void *stream) {
  fluxbin_status st = check_paged(batch);
  if (st) return st;
  const fluxbin_paged_batch &b = *batch;
  if (!(scale > 0.0f) || scale > 1.0e30f) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "scale = %g (positive, at most 1e30)", (double)scale);
  if (window < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "window = %d is negative", window);
  if (b.tokens == 0 || b.seqs == 0) return ok();
  if ((st = check_rows("q", q, ldq, (int64_t)b.heads * b.dim))) return st;
  if ((st = check_rows("out", out, ldo, (int64_t)b.heads * b.dim))) return st;
  if ((q != out || ldq != ldo) && rows_overlap(q, ldq, out, ldo, b.tokens, (int64_t)b.heads * b.dim, 2))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "out overlaps q without being it");
  if (!aligned(lse, 4)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "lse is not aligned to its elements");
  const Plan p = plan_of(b, window);
  const int64_t grid = p.tiles * b.kv_heads * std::max<int64_t>(p.splits, p.balanced ? gather_blocks(b.dim) : 1);
  if (grid > kMaxGrid) return fail(FLUXBIN_ERR_UNSUPPORTED, "%lld workgroups are beyond one launch", (long long)grid);
  const size_t need = ws_bytes(b, p);
  if (need && (!workspace || workspace_bytes < need))
    return fail(FLUXBIN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : (size_t)0);
  if (need && !aligned(workspace, 16)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "workspace not 16-byte aligned");
  AttentionArgs a{};
  a.b = paged_of(b);
  a.q = (const uint16_t *)q;
  a.out = (uint16_t *)out;
  a.lse = lse;
  a.before = (int32_t *)workspace;
  a.part = (float *)((char *)workspace + before_bytes(p));
  a.stats = a.part + p.parts * b.dim;
  a.ldq = ldq;
  a.ldo = ldo;
  a.group = b.heads / b.kv_heads;
  a.window = window;
  a.splits = p.splits;
  a.tiles = (int32_t)p.tiles;
  a.workgroups = p.shares;
  a.c = scale * 1.44269504088896340736f;
  hipStream_t s = (hipStream_t)stream;
  if (b.dtype == FLUXBIN_DT_F16) run<F16>(a, p, s);
  else run<BF16>(a, p, s);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "paged attention launch") : ok();
}

}  // extern "C"
