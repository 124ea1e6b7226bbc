// logprobs.hip -- fluxbin_token_logprobs: argument checks, the split of the rows
// over workgroups, the launches.
#include <algorithm>

#include "logprob_kernels.hpp"
#include "status.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kTargetGroups = 1024;
constexpr int64_t kFewRows = 256;  // one per CU
constexpr int32_t kTinyTop = 32;
constexpr int64_t kMaxRows = (int64_t)1 << 22;
constexpr int64_t kMaxVocab = (int64_t)1 << 28;
constexpr int64_t kMaxSplitsPerRow = 128;

struct LpPlan {
  int32_t threads, splits, split_len;
};

// Up to kFewRows rows that kLpFew threads hold in registers get one workgroup
// each and need no join: against splits and a join 1 x 5000 fp16 takes 6.3 us
// for 8.5, 1 x 32000 9.3 for 9.2, 64 x 32000 fp32 10.5 for 12.0, 256 x 32000
// 13.4 for 17.4; with two such workgroups on a CU the gain ends (400 x 32000
// fp32 25.7 for 24.4, 512 x 8000 18.0 for 15.6).
// Other rows are split, where they are few, until about kTargetGroups workgroups
// of kLpMany threads result (64 x 131072 by one workgroup of kLpFew threads per
// row takes 26.2 us, by splits 17.3), a split taking at least one step of
// kLpSmall columns; all splits are equally long (but for whole 64 columns), so
// that none is too short for a close bound of its best.
// Rows of at most kLpTinyCols columns go to one wave each, without barriers to
// wait at: 12837 x 257 fp16 9.8 us for 26.0 with 256 threads, with 20 best 20.5
// for 53.5, 32 best 22.9 for 55.3; 73 x 320, 20 best, 6.0 for 6.5; one row about
// the same. More alternatives than kTinyTop leave the bound, the least of 64
// maxima, too low (12837 x 500 with 64 best: 120 us, 256 threads 68; 73 x 320
// with 40 best 8.1, 256 threads 7.4).
LpPlan plan_of(int64_t rows, int64_t vocab, int32_t top_k) {
  if (rows <= kFewRows && vocab > kLpSmall && vocab <= kLpFewCols) return LpPlan{kLpFew, 1, (int32_t)(cdiv(vocab, 64) * 64)};
  if (vocab <= kLpTinyCols && top_k <= kTinyTop) return LpPlan{kLpTiny, 1, (int32_t)(cdiv(vocab, 64) * 64)};
  const int64_t steps = cdiv(vocab, kLpSmall);
  int64_t splits = rows > 0 ? std::max<int64_t>(1, kTargetGroups / rows) : 1;
  splits = std::min<int64_t>({splits, steps, kMaxSplitsPerRow});
  const int64_t per = cdiv(steps, splits);
  LpPlan p{kLpMany, 1, 0};
  p.split_len = (int32_t)(cdiv(cdiv(vocab, cdiv(steps, per)), 64) * 64);
  p.splits = (int32_t)cdiv(vocab, p.split_len);
  return p;
}

fluxbin_status check_shape(int64_t rows, int64_t vocab, int32_t top_k) {
  if (rows < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rows = %lld is negative", (long long)rows);
  if (vocab < 1) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "vocab = %lld (must be >= 1)", (long long)vocab);
  if (rows > kMaxRows || vocab > kMaxVocab) return fail(FLUXBIN_ERR_UNSUPPORTED, "rows above 2^22 or vocab above 2^28");
  if (top_k < 0 || top_k > vocab)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "top_k = %d outside [0, vocab = %lld]", top_k, (long long)vocab);
  if (top_k > kLpMaxTop) return fail(FLUXBIN_ERR_UNSUPPORTED, "top_k = %d (at most %d)", top_k, kLpMaxTop);
  return FLUXBIN_OK;
}

size_t ws_bytes(int64_t rows, const LpPlan &p, int32_t top_k) {
  return p.splits > 1 ? (size_t)(rows * p.splits * lp_part_bytes(top_k)) : 0;
}

template <typename E>
void launch(const LogprobArgs &a, int threads, hipStream_t st) {
  const dim3 grid((unsigned)(a.rows * a.splits)), block(threads);
  if (threads == kLpFew) hipLaunchKernelGGL((logprob_rows_kernel<E, false, kLpFew>), grid, block, 0, st, a);
  else if (threads == kLpTiny) hipLaunchKernelGGL((logprob_rows_kernel<E, true, kLpTiny>), grid, block, 0, st, a);
  else if (a.split_len <= kLpSmall) hipLaunchKernelGGL((logprob_rows_kernel<E, true, kLpMany>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((logprob_rows_kernel<E, false, kLpMany>), grid, block, 0, st, a);
  if (a.splits > 1) hipLaunchKernelGGL(logprob_join_kernel<E>, dim3((unsigned)a.rows), dim3(kLpMany), 0, st, a);
}

}  // namespace

extern "C" {

fluxbin_status fluxbin_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int32_t top_k, size_t *bytes) {
  const fluxbin_status st = check_shape(rows, vocab, top_k);
  if (st) return st;
  if (!bytes) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = ws_bytes(rows, plan_of(rows, vocab, top_k), top_k);
  return ok();
}

fluxbin_status fluxbin_token_logprobs(const void *logits, int64_t ld, int32_t dtype, int64_t rows, int64_t vocab,
                                      float logit_scale, const int64_t *targets, float *logprob, float *entropy,
                                      int32_t top_k, float *top_logprob, int64_t *top_index, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  if (dtype != FLUXBIN_DT_F16 && dtype != FLUXBIN_DT_BF16 && dtype != FLUXBIN_DT_F32)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "dtype = %d (fp16, bf16 or fp32)", dtype);
  const fluxbin_status st = check_shape(rows, vocab, top_k);
  if (st) return st;
  if (!(logit_scale > 0.0f) || logit_scale > 1.0e30f)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "logit_scale = %g (positive, at most 1e30)", (double)logit_scale);
  if (!targets != !logprob) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "targets and logprob go together");
  if (!targets && !entropy && !top_k) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "nothing to write");
  if (rows == 0) return ok();
  if (!logits) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "logits is NULL");
  if (top_k && (!top_logprob || !top_index)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "top_k without top_logprob and top_index");
  if (ld < vocab) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "ld = %lld < vocab = %lld", (long long)ld, (long long)vocab);
  if (!aligned(logits, dtype == FLUXBIN_DT_F32 ? 4 : 2) || !aligned(targets, 8) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || (top_k && (!aligned(top_logprob, 4) || !aligned(top_index, 8))))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "a pointer is not aligned to its elements");
  const LpPlan p = plan_of(rows, vocab, top_k);
  const size_t need = ws_bytes(rows, p, top_k);
  if (need && (!workspace || workspace_bytes < need))
    return fail(FLUXBIN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : (size_t)0);
  if (need && !aligned(workspace, 16)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "workspace not 16-byte aligned");
  LogprobArgs a{};
  a.logits = logits;
  a.targets = targets;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_logprob = top_logprob;
  a.top_index = top_index;
  a.workspace = (uint8_t *)workspace;
  a.rows = rows;
  a.ld = ld;
  a.vocab = (int32_t)vocab;
  a.top_k = top_k;
  a.splits = p.splits;
  a.split_len = p.split_len;
  a.scale = logit_scale;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == FLUXBIN_DT_F16) launch<F16>(a, p.threads, s);
  else if (dtype == FLUXBIN_DT_BF16) launch<BF16>(a, p.threads, s);
  else launch<F32>(a, p.threads, s);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "token logprobs launch") : ok();
}

}  // extern "C"
