// act_ops.hip -- fluxbin_quantize_rows and fluxbin_add_rmsnorm: argument checks,
// the choice of a kernel instance, the launch.
#include <algorithm>

#include "act_kernels.hpp"
#include "status.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 30;
constexpr int64_t kMaxGrid = (int64_t)1 << 20;

int elem_bytes(int32_t dtype) { return dtype == FLUXBIN_DT_F32 ? 4 : 2; }

fluxbin_status check_shape(int32_t dtype, int64_t rows, int64_t cols) {
  if (dtype != FLUXBIN_DT_F16 && dtype != FLUXBIN_DT_BF16 && dtype != FLUXBIN_DT_F32)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "dtype = %d (fp16, bf16 or fp32)", dtype);
  if (rows < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "rows = %lld is negative", (long long)rows);
  if (cols < 1) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "cols = %lld (must be >= 1)", (long long)cols);
  if (cols > kMaxCols) return fail(FLUXBIN_ERR_UNSUPPORTED, "cols = %lld above 2^30", (long long)cols);
  return FLUXBIN_OK;
}

// One matrix argument: its pointer, natural alignment and row stride.
fluxbin_status check_matrix(const char *name, const void *p, int64_t ld, int64_t cols, int bytes) {
  if (!p) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (!aligned(p, bytes)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "%s is not aligned to its %d-byte elements", name, bytes);
  if (ld < cols)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "the row stride of %s, %lld, is below cols = %lld", name, (long long)ld,
                (long long)cols);
  return FLUXBIN_OK;
}

template <typename E, bool NORM, int TPR, int U>
void launch_rows(const ActArgs &a, hipStream_t st) {
  constexpr int TPB = TPR < 256 ? 256 : TPR;
  const int64_t grid = std::min(cdiv(a.rows, TPB / TPR), kMaxGrid);
  hipLaunchKernelGGL((act_rows_kernel<E, NORM, TPR, U>), dim3((unsigned)grid), dim3(TPB), 0, st, a);
}

// The fewest threads that hold a row in two units each (fewer, later stores
// overlap more rows' loads), measured on fp16 rows: 8192 x 1024 15.6 us with one
// wave and two units, 18.9 with four waves and one; 8192 x 2048 23.7 with four
// waves, 34 with eight; 4096 x 4096 24.4 / 25.5 / 34.6 with 256 x 2, 512 x 1,
// 1024 x 1; 8192 x 8192 84 / 92 with 512 x 2, 1024 x 1.  Up to 16384 columns the
// norm, with three units per eight elements, takes 1024 x 2 (2000 x 16384: 54
// us, 512 x 4 64), the quantisation 512 x 4 (8000 x 11008: 51 us, 1024 x 2 60).
template <typename E, bool NORM>
void launch_act(const ActArgs &a, hipStream_t st) {
  const int64_t units = cdiv(a.cols, kUnit);
  const dim3 rows((unsigned)std::min(a.rows, kMaxGrid));
  if (a.cols < kUnit) hipLaunchKernelGGL((act_long_rows_kernel<E, NORM, true>), rows, dim3(1024), 0, st, a);
  else if (units > 4096) hipLaunchKernelGGL((act_long_rows_kernel<E, NORM, false>), rows, dim3(1024), 0, st, a);
  else if (units <= 64) launch_rows<E, NORM, 64, 1>(a, st);
  else if (units <= 128) launch_rows<E, NORM, 64, 2>(a, st);
  else if (units <= 256) launch_rows<E, NORM, 256, 1>(a, st);
  else if (units <= 512) launch_rows<E, NORM, 256, 2>(a, st);
  else if (units <= 1024) launch_rows<E, NORM, 512, 2>(a, st);
  else if (units <= 2048) launch_rows<E, NORM, NORM ? 1024 : 512, NORM ? 2 : 4>(a, st);
  else launch_rows<E, NORM, 1024, 4>(a, st);
}

template <bool NORM>
fluxbin_status run(const ActArgs &a, int32_t dtype, void *stream, const char *what) {
  hipStream_t st = (hipStream_t)stream;
  if (dtype == FLUXBIN_DT_F16) launch_act<F16, NORM>(a, st);
  else if (dtype == FLUXBIN_DT_BF16) launch_act<BF16, NORM>(a, st);
  else launch_act<F32, NORM>(a, st);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, what) : ok();
}

}  // namespace

extern "C" {

fluxbin_status fluxbin_quantize_rows(const void *x, int64_t ldx, int32_t dtype, int64_t rows, int64_t cols, int8_t *q,
                                     int64_t ldq, float *scale, void *stream) {
  fluxbin_status st = check_shape(dtype, rows, cols);
  if (st) return st;
  if (rows == 0) return ok();
  if ((st = check_matrix("x", x, ldx, cols, elem_bytes(dtype)))) return st;
  if ((st = check_matrix("q", q, ldq, cols, 1))) return st;
  if ((st = check_matrix("scale", scale, 1, 1, 4))) return st;
  ActArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  a.rows = rows;
  a.cols = cols;
  return run<false>(a, dtype, stream, "row quantisation launch");
}

fluxbin_status fluxbin_add_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                                   int32_t dtype, int64_t rows, int64_t cols, float eps, void *residual_out, int64_t ldro,
                                   void *y, int64_t ldy, int8_t *q, int64_t ldq, float *scale, void *stream) {
  fluxbin_status st = check_shape(dtype, rows, cols);
  if (st) return st;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "eps = %g (finite, >= 0)", (double)eps);
  if (!y && !q) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "y and q are both NULL: nothing to write");
  if (residual_out && !residual) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "residual_out without residual");
  if (rows == 0) return ok();
  const int b = elem_bytes(dtype);
  if ((st = check_matrix("x", x, ldx, cols, b))) return st;
  if (residual && (st = check_matrix("residual", residual, ldr, cols, b))) return st;
  if ((st = check_matrix("weight", weight, cols, cols, b))) return st;
  if (residual_out && (st = check_matrix("residual_out", residual_out, ldro, cols, b))) return st;
  if (y && (st = check_matrix("y", y, ldy, cols, b))) return st;
  if (q && (st = check_matrix("q", q, ldq, cols, 1))) return st;
  if (q && (st = check_matrix("scale", scale, 1, 1, 4))) return st;
  ActArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.residual = residual;
  a.ldr = ldr;
  a.weight = weight;
  a.residual_out = residual_out;
  a.ldro = ldro;
  a.y = y;
  a.ldy = ldy;
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.inv_cols = 1.0f / (float)cols;
  return run<true>(a, dtype, stream, "norm launch");
}

}  // extern "C"
