// rope_append.hip -- fluxbin_rope_append: argument checks, the choice of a kernel
// instance, the launch.
#include <algorithm>

#include "rope_kernels.hpp"

using namespace fluxbin;

namespace {

// Runs of 16 bytes where dim and rotary_dim are made of pairs of them.
int run_elems(int64_t dim, int64_t rot) { return dim % 16 == 0 && rot % 16 == 0 ? 8 : 4; }

// Lanes to a row, two runs each.
int row_lanes(int64_t dim, int run) {
  int lanes = 4;
  while (2 * run * lanes < dim) lanes *= 2;
  return lanes;
}

template <typename E, int C, int LPR>
void launch(const RopeArgs &a, unsigned grid, bool near, hipStream_t st) {
  const dim3 block(256);
  if (a.q_norm || a.k_norm) hipLaunchKernelGGL((rope_append_kernel<E, C, LPR, true>), dim3(grid), block, 0, st, a, near);
  else hipLaunchKernelGGL((rope_append_kernel<E, C, LPR, false>), dim3(grid), block, 0, st, a, near);
}

template <typename E>
void run(const RopeArgs &a, unsigned grid, int elems, int lanes, bool near, hipStream_t st) {
  if (elems == 8 && lanes == 4) launch<E, 8, 4>(a, grid, near, st);
  else if (elems == 8 && lanes == 8) launch<E, 8, 8>(a, grid, near, st);
  else if (elems == 8) launch<E, 8, 16>(a, grid, near, st);
  else if (lanes == 4) launch<E, 4, 4>(a, grid, near, st);
  else if (lanes == 8) launch<E, 4, 8>(a, grid, near, st);
  else if (lanes == 16) launch<E, 4, 16>(a, grid, near, st);
  else launch<E, 4, 32>(a, grid, near, st);
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
  if (q && q == q_out && ldq != ldqo) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "q_out is q with another stride");
  if (q && q != q_out && rows_overlap(q, ldq, q_out, ldqo, b.tokens, (int64_t)b.heads * b.dim, 2))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "q_out overlaps q without being it");
  if ((st = check_rows("k", k, ldk, (int64_t)b.kv_heads * b.dim))) return st;
  if ((st = check_rows("v", v, ldv, (int64_t)b.kv_heads * b.dim))) return st;
  if (!aligned(q_norm, 2) || !aligned(k_norm, 2) || !aligned(positions, 4) || !aligned(freq, 8))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "q_norm, k_norm, positions or freq is not aligned to its elements");
  if (rotary_dim && !freq) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rotary_dim without freq");
  const int64_t rows = (q ? b.heads : 0) + 2 * (int64_t)b.kv_heads;
  const int elems = run_elems(b.dim, rotary_dim), lanes = row_lanes(b.dim, elems);
  const int64_t runs = cdiv(rows, 64 / lanes), grid = cdiv(runs * b.tokens, 4);
  if (grid >= (int64_t)1 << 24)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "%lld tokens of %lld rows are beyond one launch", (long long)b.tokens, (long long)rows);
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
  a.runs = (int32_t)runs;
  hipStream_t s = (hipStream_t)stream;
  if (b.dtype == FLUXBIN_DT_F16) run<F16>(a, (unsigned)grid, elems, lanes, pairs == FLUXBIN_ROPE_NEAR, s);
  else run<BF16>(a, (unsigned)grid, elems, lanes, pairs == FLUXBIN_ROPE_NEAR, s);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "rope append launch") : ok();
}
