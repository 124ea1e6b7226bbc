// gemm_w8a8.hip -- fluxbin_gemm_w8a8: argument checks, the choice of a kernel
// instance, the launch.
#include "gemm_w8a8_kernel.hpp"
#include "status.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kMaxK = 131071;            // 131071 * 128 * 128 < 2^31
constexpr int64_t kMaxMN = (int64_t)1 << 27;
constexpr int64_t kTileStride = (int64_t)1 << 23;  // 256 strides stay below 2^31 (32-bit offsets)

template <typename E, int BN, int BM, int WN, int WM, int S, int G>
void launch_tile(const GemmArgs &g, hipStream_t st) {
  hipLaunchKernelGGL((gemm_w8a8_tile_kernel<E, BN, BM, WN, WM, S, G>), dim3((unsigned)(cdiv(g.n, BN) * cdiv(g.m, BM))),
                     dim3(64 * WN * WM), 0, st, g);
}

template <typename E>
void launch(const GemmArgs &g, hipStream_t st) {
  const unsigned nb = (unsigned)cdiv(g.n, 16);
  if (g.m <= 16) hipLaunchKernelGGL((gemm_w8a8_rows_kernel<E, 1, 4>), dim3(nb, 1), dim3(256), 0, st, g);
  else if (g.m <= 64 || g.lda > kTileStride || g.ldw > kTileStride)
    hipLaunchKernelGGL((gemm_w8a8_rows_kernel<E, 4, 4>), dim3(nb, (unsigned)cdiv(g.m, 64)), dim3(256), 0, st, g);
  else if (g.m <= 1024) launch_tile<E, 64, 64, 2, 2, 4, 4>(g, st);
  else launch_tile<E, 256, 256, 2, 4, 2, 1>(g, st);
}

}  // namespace

extern "C" fluxbin_status fluxbin_gemm_w8a8(const int8_t *a, int64_t lda, const float *a_scale, const int8_t *w,
                                            int64_t ldw, const float *w_scale, const float *bias, int64_t m, int64_t n,
                                            int64_t k, void *y, int64_t ldy, int32_t dtype, void *stream) {
  if (dtype != FLUXBIN_DT_F16 && dtype != FLUXBIN_DT_BF16 && dtype != FLUXBIN_DT_F32)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "dtype = %d (fp16, bf16 or fp32)", dtype);
  if (m < 0 || n < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "m = %lld, n = %lld (negative)", (long long)m, (long long)n);
  if (k < 1) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "k = %lld (must be >= 1)", (long long)k);
  if (k > kMaxK) return fail(FLUXBIN_ERR_UNSUPPORTED, "k = %lld above %lld: the sums could leave int32", (long long)k,
                             (long long)kMaxK);
  if (m > kMaxMN || n > kMaxMN) return fail(FLUXBIN_ERR_UNSUPPORTED, "m or n above 2^27");
  if (m == 0 || n == 0) return ok();
  if (!a || !a_scale || !w || !w_scale || !y) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "NULL pointer");
  if (!aligned(a, 16) || !aligned(w, 16)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "a and w must be 16-byte aligned");
  const int64_t kp = cdiv(k, 16) * 16;
  if (lda % 16 || ldw % 16 || lda < kp || ldw < kp)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "lda = %lld, ldw = %lld: multiples of 16, at least k rounded up to one (%lld)",
                (long long)lda, (long long)ldw, (long long)kp);
  if (!aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "scales and bias must be 4-byte aligned");
  if (!aligned(y, dtype == FLUXBIN_DT_F32 ? 4 : 2))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "y is not aligned to its elements");
  if (ldy < n) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "ldy = %lld < n = %lld", (long long)ldy, (long long)n);
  GemmArgs g{a, w, a_scale, w_scale, bias, y, lda, ldw, ldy, (int32_t)m, (int32_t)n, (int32_t)k};
  hipStream_t st = (hipStream_t)stream;
  if (dtype == FLUXBIN_DT_F16) launch<F16>(g, st);
  else if (dtype == FLUXBIN_DT_BF16) launch<BF16>(g, st);
  else launch<F32>(g, st);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? hip_fail(e, "gemm_w8a8 launch") : ok();
}
