// rope_append.hip -- fluxbin_rope_append: argument checks, the choice of a kernel
// instance, the launch.
#include <algorithm>

#include "rope_kernels.hpp"

using namespace fluxbin;

namespace {

template <typename E, int C, int LPR>
void launch(const RopeArgs &a, int rows, bool near, hipStream_t st) {
  RopeArgs b = a;
  b.runs = (int32_t)cdiv(rows, 64 / LPR);
  const dim3 grid((unsigned)cdiv(b.runs * (int64_t)a.b.tokens, 4)), block(256);
  if (a.q_norm || a.k_norm) hipLaunchKernelGGL((rope_append_kernel<E, C, LPR, true>), grid, block, 0, st, b, near);
  else hipLaunchKernelGGL((rope_append_kernel<E, C, LPR, false>), grid, block, 0, st, b, near);
}

template <typename E, int C>
void with_lanes(const RopeArgs &a, int rows, bool near, hipStream_t st) {
  if (a.b.dim <= 8 * C) launch<E, C, 4>(a, rows, near, st);
  else if (a.b.dim <= 16 * C) launch<E, C, 8>(a, rows, near, st);
  else if (C == 8 || a.b.dim <= 32 * C) launch<E, C, 16>(a, rows, near, st);
  else launch<E, C, C == 8 ? 16 : 32>(a, rows, near, st);
}

template <typename E>
void run(const RopeArgs &a, int rows, bool near, hipStream_t st) {
  if (a.b.dim % 16 == 0 && a.rot % 16 == 0) with_lanes<E, 8>(a, rows, near, st);
  else with_lanes<E, 4>(a, rows, near, st);
}

}  // namespace

extern "C" fluxbin_status fluxbin_rope_append(const fluxbin_paged_batch *batch, const void *q, int64_t ldq, const void *k,
                                              int64_t ldk, const void *v, int64_t ldv, const void *q_norm, const void *k_norm,
                                              float eps, const double *freq, int32_t rotary_dim, int32_t pairs,
                                              float rope_scale, const int32_t *positions, void *q_out, int64_t ldqo,
                                              void *stream) {
  fluxbin_status st = check_paged(batch);
  if (st) return st;
  const fluxbin_paged_batch &b = *batch;
  if (rotary_dim < 0 || rotary_dim > b.dim || rotary_dim % 8)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rotary_dim = %d (a multiple of 8 in [0, dim = %d])", rotary_dim, b.dim);
  if (pairs != FLUXBIN_ROPE_HALF && pairs != FLUXBIN_ROPE_NEAR) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "pairs = %d", pairs);
  if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "eps = %g (finite, >= 0)", (double)eps);
  if (!(rope_scale >= -3.0e38f && rope_scale <= 3.0e38f))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rope_scale = %g is not finite", (double)rope_scale);
  if (!q != !q_out) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "q and q_out go together");
  if (b.tokens == 0 || b.seqs == 0) return ok();
  if (q && (st = check_rows("q", q, ldq, (int64_t)b.heads * b.dim))) return st;
  if (q && (st = check_rows("q_out", q_out, ldqo, (int64_t)b.heads * b.dim))) return st;
  if ((st = check_rows("k", k, ldk, (int64_t)b.kv_heads * b.dim))) return st;
  if ((st = check_rows("v", v, ldv, (int64_t)b.kv_heads * b.dim))) return st;
  if (!aligned(q_norm, 2) || !aligned(k_norm, 2) || !aligned(positions, 4) || !aligned(freq, 8))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "q_norm, k_norm, positions or freq is not aligned to its elements");
  if (rotary_dim && !freq) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rotary_dim without freq");
  RopeArgs a{};
  a.b = paged_of(b);
  a.q = (const uint16_t *)q;
  a.k = (const uint16_t *)k;
  a.v = (const uint16_t *)v;
  a.q_norm = (const uint16_t *)q_norm;
  a.k_norm = (const uint16_t *)k_norm;
  a.q_out = (uint16_t *)q_out;
  a.freq = freq;
  a.positions = positions;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldqo = ldqo;
  a.rot = rotary_dim;
  a.eps = eps;
  a.inv_dim = 1.0f / (float)b.dim;
  a.scale = rope_scale;
  const int rows = (q ? b.heads : 0) + 2 * b.kv_heads;
  hipStream_t s = (hipStream_t)stream;
  if (b.dtype == FLUXBIN_DT_F16) run<F16>(a, rows, pairs == FLUXBIN_ROPE_NEAR, s);
  else run<BF16>(a, rows, pairs == FLUXBIN_ROPE_NEAR, s);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "rope append launch") : ok();
}
