// paged_attention.hip -- fluxbin_paged_attention: argument checks, the choice of a
// kernel and of the split of the keys, the launches.
#include <algorithm>

#include "attention_kernels.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kTargetGroups = 256;  // one to a CU
constexpr int64_t kMinKeys = 512;       // of a split
constexpr int64_t kMaxSplits = 64;      // the join's lanes
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;

struct Plan {
  int32_t rows, splits;  // rows of a workgroup
  int64_t tiles;
};

// Sequences whose new tokens fill at most 32 rows of a key head on average go to
// the kernel whose waves share the rows and split the keys.  Where the tiles are
// fewer than kTargetGroups, the keys are split over workgroups too.
Plan plan_of(const fluxbin_paged_batch &b, int64_t window) {
  const int64_t group = b.heads / b.kv_heads, per_seq = b.seqs ? cdiv(b.tokens * group, b.seqs) : 0;
  Plan p{};
  p.rows = per_seq <= 32 ? 32 : 128;
  p.tiles = b.tokens * group / p.rows + b.seqs;
  const int64_t cap = b.table_pages * b.page_size, most = b.max_kv_len ? std::min(b.max_kv_len, cap) : cap;
  const int64_t keys = window ? std::min(most, window + b.tokens) : most;
  const int64_t busy = std::max<int64_t>(1, b.seqs * cdiv(per_seq, p.rows) * b.kv_heads);
  p.splits = (int32_t)std::max<int64_t>(1, std::min({kTargetGroups / busy, cdiv(keys, kMinKeys), kMaxSplits}));
  return p;
}

size_t ws_bytes(const fluxbin_paged_batch &b, const Plan &p) {
  return p.splits > 1 ? (size_t)(b.tokens * b.heads * p.splits * (b.dim + 2)) * 4 : 0;
}

template <typename E, int D>
void launch(const AttentionArgs &a, const Plan &p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.splits * a.b.kv_heads));
  if (p.rows == 32) hipLaunchKernelGGL((attention_few_kernel<E, D>), grid, dim3(64 * Few<D>::W), 0, st, a);
  else hipLaunchKernelGGL((attention_chunk_kernel<E, D, 1>), grid, dim3(256), 0, st, a);
  if (p.splits > 1)
    hipLaunchKernelGGL(attention_join_kernel<E>, dim3((unsigned)cdiv((int64_t)a.b.tokens * a.b.heads, 4)), dim3(256), 0, st, a);
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
  *bytes = ws_bytes(*batch, plan_of(*batch, 0));
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
  if (!aligned(lse, 4)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "lse is not aligned to its elements");
  const Plan p = plan_of(b, window);
  const int64_t grid = p.tiles * p.splits * b.kv_heads;
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
  a.part = (float *)workspace;
  a.ldq = ldq;
  a.ldo = ldo;
  a.parts = b.tokens * b.heads * p.splits;
  a.group = b.heads / b.kv_heads;
  a.window = window;
  a.splits = p.splits;
  a.tiles = (int32_t)p.tiles;
  a.c = scale * 1.44269504088896340736f;
  hipStream_t s = (hipStream_t)stream;
  if (b.dtype == FLUXBIN_DT_F16) run<F16>(a, p, s);
  else run<BF16>(a, p, s);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "paged attention launch") : ok();
}

}  // extern "C"
