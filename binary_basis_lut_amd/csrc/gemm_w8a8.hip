// gemm_w8a8.hip -- fluxbin_gemm_w8a8: argument checks, the choice of a kernel
// instance, the launch.
#include <algorithm>

#include "gemm_w8a8_kernel.hpp"
#include "status.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kMaxK = 131071;            // 131071 * 128 * 128 < 2^31
constexpr int64_t kMaxMN = (int64_t)1 << 27;
constexpr int64_t kTileStride = (int64_t)1 << 23;  // 256 strides stay below 2^31 (32-bit offsets)

template <typename E, int BN, int BM, int WN, int WM, int WK, int KB, int S, int G>
void launch_tile(const GemmArgs &g, hipStream_t st) {
  hipLaunchKernelGGL((gemm_w8a8_tile_kernel<E, BN, BM, WN, WM, WK, KB, S, G>),
                     dim3((unsigned)(cdiv(g.n, BN) * cdiv(g.m, BM))), dim3(64 * WN * WM * WK), 0, st, g);
}

// Which tile: a workgroup's time is taken as the larger of its loads, at the 55
// GB/s that one CU sustains on rows that come from HBM and the Infinity Cache,
// and its products, at the 9 TOP/s of a CU (2.3 POP/s in all), and the CUs take
// ceil(tiles / 256) workgroups one after another.  Measured (k x n = 4096 x 4096
// unless said; us for the tiles 32 x 32, 32 x 64, 64 x 64, 64 x 128, 128 x 128,
// 256 x 256, channels x tokens):
//   64 tokens     8.6 / 10.4 / 13.0 / - / - / -
//   128 tokens    - / 10.4 / 13.2 / 16.9 / - / -
//   1024 tokens   - / - / - / 34.8 / 27.3 / 57.2
//   64 tokens, 11008 x 16384     54.5 / - / 47.8 / - / - / -
//   333 tokens, 11008 x 4096     - / - / 43.9 / 38.4 / 51.6 / -
//   8192 tokens, 8192 x 28672    - / - / - / - / 2480 / 1850
struct Tile {
  int bn, bm;
};
constexpr Tile kTiles[] = {{32, 32}, {32, 64}, {64, 64}, {64, 128}, {128, 128}, {256, 256}};

int pick_tile(const GemmArgs &g) {
  int best = 0;
  double least = 0;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile &t = kTiles[i];
    const double rounds = (double)cdiv(cdiv(g.n, t.bn) * cdiv(g.m, t.bm), 256);
    const double cost = rounds * std::max((t.bn + t.bm) / 55e9, 2.0 * t.bn * t.bm / 9e12);
    if (i == 0 || cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

template <typename E>
void launch(const GemmArgs &g, hipStream_t st) {
  // Up to 16 tokens each channel's weights go straight to registers: one token
  // at 4096 x 4096 5.6 us (32 x 32 tiles: 7.6), at 8192 x 28672 40 (45), 16 tokens
  // at 4096 x 4096 6.5 (7.9); but 16 tokens over 32000 channels 35 (31): there the
  // tokens, read again by every 16 channels, cost as much as the weights.
  if (g.m <= 4 || (g.m <= 16 && g.n <= 16384) || g.lda > kTileStride || g.ldw > kTileStride) {
    hipLaunchKernelGGL((gemm_w8a8_rows_kernel<E, 8>), dim3((unsigned)cdiv(g.n, 16), (unsigned)cdiv(g.m, 16)), dim3(512), 0,
                       st, g);
    return;
  }
  switch (pick_tile(g)) {
    case 0: launch_tile<E, 32, 32, 1, 1, 4, 256, 4, 2>(g, st); break;
    case 1: launch_tile<E, 32, 64, 1, 2, 2, 256, 4, 4>(g, st); break;
    case 2: launch_tile<E, 64, 64, 2, 2, 1, 128, 4, 4>(g, st); break;
    case 3: launch_tile<E, 64, 128, 2, 4, 1, 128, 4, 4>(g, st); break;
    case 4: launch_tile<E, 128, 128, 2, 4, 1, 128, 4, 2>(g, st); break;
    default: launch_tile<E, 256, 256, 2, 4, 1, 128, 2, 1>(g, st); break;
  }
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
