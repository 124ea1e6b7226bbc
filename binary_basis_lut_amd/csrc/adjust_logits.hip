// adjust_logits.hip -- fluxbin_adjust_logits: argument checks and the launch.
#include "adjust_kernels.hpp"
#include "status.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 22, kMaxVocab = (int64_t)1 << 28, kMaxHistory = ((int64_t)1 << 30) - 1, kMaxBiases = 4096;

constexpr int64_t kShort = 4096;  // tokens of a row that one workgroup of 256 threads takes

int64_t slice_of(int64_t vocab, int64_t biases) { return vocab <= kShort ? kShort : biases ? 8192 : 16384; }

template <typename E, bool BIAS, bool TINY, int T, int SLICE>
void launch(const AdjustArgs &a, hipStream_t st) {
  hipLaunchKernelGGL((adjust_logits_kernel<E, BIAS, TINY, T, SLICE>), dim3((unsigned)(a.rows * a.slices)), dim3(T), 0, st, a);
}

template <typename E>
void run(const AdjustArgs &a, hipStream_t st) {
  if (a.vocab < kUnit && a.biases) launch<E, true, true, 256, kShort>(a, st);
  else if (a.vocab < kUnit) launch<E, false, true, 256, kShort>(a, st);
  else if (a.vocab <= kShort && a.biases) launch<E, true, false, 256, kShort>(a, st);
  else if (a.vocab <= kShort) launch<E, false, false, 256, kShort>(a, st);
  else if (a.biases) launch<E, true, false, 1024, 8192>(a, st);
  else launch<E, false, false, 1024, 16384>(a, st);
}

}  // namespace

extern "C" fluxbin_status fluxbin_adjust_logits(const void *logits, int64_t ld, int32_t dtype, int64_t rows, int64_t vocab,
                                                const int32_t *history, int64_t ldh, int64_t history_cols,
                                                const int32_t *prompt_len, const int32_t *total_len, const float *repetition,
                                                const float *frequency, const float *presence, const int32_t *bias_index,
                                                const float *bias_value, int64_t ldb, int64_t biases, const uint32_t *mask,
                                                int64_t ldm, void *out, int64_t ldo, void *stream) {
  if (dtype != FLUXBIN_DT_F16 && dtype != FLUXBIN_DT_BF16 && dtype != FLUXBIN_DT_F32)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "dtype = %d (fp16, bf16 or fp32)", dtype);
  if (rows < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rows = %lld is negative", (long long)rows);
  if (vocab < 1) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "vocab = %lld (must be >= 1)", (long long)vocab);
  if (rows > kMaxRows || vocab > kMaxVocab) return fail(FLUXBIN_ERR_UNSUPPORTED, "rows above 2^22 or vocab above 2^28");
  if (history_cols < 0 || biases < 0)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "history_cols = %lld, biases = %lld", (long long)history_cols, (long long)biases);
  if (history_cols > kMaxHistory || biases > kMaxBiases)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "history_cols from 2^30 on or more than %lld biases", (long long)kMaxBiases);
  if (rows == 0) return ok();
  const int bytes = dtype == FLUXBIN_DT_F32 ? 4 : 2;
  const int64_t slices = cdiv(vocab, slice_of(vocab, biases));
  if (rows * slices >= (int64_t)1 << 22)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "%lld rows of %lld tokens are beyond one launch", (long long)rows, (long long)vocab);
  if (!logits || !out) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "logits or out is NULL");
  if (ld < vocab || ldo < vocab)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "ld = %lld or ldo = %lld below vocab = %lld", (long long)ld, (long long)ldo, (long long)vocab);
  if (logits == out && ld != ldo) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "out is logits with another stride");
  if (logits != out && rows_overlap(logits, ld, out, ldo, rows, vocab, bytes))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "out overlaps logits without being them");
  if (history_cols && !history) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "history_cols without history");
  if (history && ldh < history_cols)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "ldh = %lld < history_cols = %lld", (long long)ldh, (long long)history_cols);
  if (biases && (!bias_index || !bias_value)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "biases without bias_index and bias_value");
  if (biases && ldb < biases) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "ldb = %lld < biases = %lld", (long long)ldb, (long long)biases);
  if (mask && ldm < cdiv(vocab, 32)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "ldm = %lld words below vocab / 32", (long long)ldm);
  if (!aligned(logits, bytes) || !aligned(out, bytes) || !aligned(history, 4) || !aligned(prompt_len, 4) || !aligned(total_len, 4) ||
      !aligned(repetition, 4) || !aligned(frequency, 4) || !aligned(presence, 4) || !aligned(bias_index, 4) ||
      !aligned(bias_value, 4) || !aligned(mask, 4))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "a pointer is not aligned to its elements");
  AdjustArgs a{};
  a.logits = logits;
  a.out = out;
  a.history = history_cols ? history : nullptr;
  a.prompt_len = prompt_len;
  a.total_len = total_len;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_index = bias_index;
  a.bias_value = bias_value;
  a.mask = mask;
  a.ld = ld;
  a.ldo = ldo;
  a.ldh = ldh;
  a.ldb = ldb;
  a.ldm = ldm;
  a.rows = rows;
  a.vocab = (int32_t)vocab;
  a.history_cols = (int32_t)history_cols;
  a.biases = (int32_t)biases;
  a.slices = (int32_t)slices;
  hipStream_t st = (hipStream_t)stream;
  if (dtype == FLUXBIN_DT_F16) run<F16>(a, st);
  else if (dtype == FLUXBIN_DT_BF16) run<BF16>(a, st);
  else run<F32>(a, st);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "logit adjustment launch") : ok();
}
