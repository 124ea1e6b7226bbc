// gemm_w8a8.hip -- fluxbin_gemm_w8a8: argument checks, the choice of a kernel
// instance, the launch.
#include <algorithm>

#include "gemm_w8a8_kernel.hpp"
#include "status.hpp"

using namespace fluxbin;

namespace {

constexpr int64_t kMaxK = 131071;            // 131071 * 128 * 128 < 2^31
constexpr int64_t kCus = 256;                // compute units of an MI355X
constexpr int64_t kMaxMN = (int64_t)1 << 27;
constexpr int64_t kTileStride = (int64_t)1 << 23;  // 256 strides stay below 2^31 (32-bit offsets)
constexpr int64_t kRowsN = (int64_t)1 << 26;       // channels and tokens of one launch of the kernel without
constexpr int64_t kRowsM = (int64_t)1 << 19;       // tiles: 2^31 threads along x, 2^15 workgroups along y

template <typename E, int BN, int BM, int WN, int WM, int WK, int KB, int S, int G>
void launch_tile(const GemmArgs &g, hipStream_t st) {
  hipLaunchKernelGGL((gemm_w8a8_tile_kernel<E, BN, BM, WN, WM, WK, KB, S, G>),
                     dim3((unsigned)(cdiv(g.n, BN) * cdiv(g.m, BM))), dim3(64 * WN * WM * WK), 0, st, g);
}

// The kernel without tiles has a workgroup for 16 channels (x) and 16 tokens (y);
// sizes beyond a grid (fewer than 2^32 threads along x, at most 65535 workgroups
// along y) take several launches.  Only strides that rule the tiles out come to that.
template <typename E>
void launch_rows(const GemmArgs &g, hipStream_t st) {
  for (int64_t m0 = 0; m0 < g.m; m0 += kRowsM)
    for (int64_t n0 = 0; n0 < g.n; n0 += kRowsN) {
      GemmArgs part = g;
      part.a += m0 * g.lda;
      part.a_scale += m0;
      part.w += n0 * g.ldw;
      part.w_scale += n0;
      if (g.bias) part.bias += n0;
      part.y = (typename E::raw *)g.y + m0 * g.ldy + n0;
      part.m = (int32_t)std::min(g.m - m0, kRowsM);
      part.n = (int32_t)std::min(g.n - n0, kRowsN);
      hipLaunchKernelGGL((gemm_w8a8_rows_kernel<E, 8>), dim3((unsigned)cdiv(part.n, 16), (unsigned)cdiv(part.m, 16)), dim3(512),
                         0, st, part);
    }
}

// Which kernel and tile (channels x tokens): a CU takes ceil(tiles / 256) of them,
// each for a fixed time (the first loads' latency, the outputs) and a time per
// column of k, both fitted to measurements.  16 x 16 is the kernel without LDS
// stages; its tokens come from the caches and cost by their number.  Tiles of
// two stages leave room for several workgroups on a CU, whose first loads and
// outputs overlap, and pay where there are more tiles than CUs; the same tiles
// with four stages keep more loads in flight where there are not.  Measured
// (us, weights from HBM; tokens x channels x k):
//                      16x16 32x32 64x32 32x64 64x64 64x128 128x128 same, two 256x256
//   1 x 4096 x 4096       5.6   7.6    -     -     -     -      -        -       -
//   1 x 57344 x 8192       74    88    -     -     -     -      -        -       -
//   16 x 8192 x 8192       19    15   20     -     -     -      -        -       -
//   16 x 32000 x 4096      36    31   28     -     -     -      -        -       -
//   64 x 4096 x 4096        -   6.9    -   9.9    13     -      -        -       -
//   64 x 16384 x 8192       -    48   42    45    33    37      -        -       -
//   128 x 16384 x 8192      -     -   63    66    49    40     49       70       -
//   333 x 4096 x 11008      -     -    -     -    43    36     51        -       -
//   200 x 57344 x 4096      -     -    -     -   119   113     98       91       -
//   1024 x 4096 x 4096      -     -    -     -     -    35     27       47      57
//   3200 x 51200 x 144      -  1045    -     -   279   286    209      132     189
//   4096 x 4096 x 512       -     -    -     -     -     -     25       21      24
//   2000 x 8192 x 2000      -     -    -     -     -     -     69       59      48
//   8192 x 28672 x 8192     -     -    -     -     -     -   2480        -    1740
struct Tile {
  int bn, bm;
  int threads;
  bool many;            // for more tiles than CUs only
  double fixed, per_k;  // us, ns
};
constexpr Tile kTiles[] = {{16, 16, 512, false, 0.3, 0.6},   {32, 32, 256, false, 0.8, 1.6},  {64, 32, 256, false, 1.0, 3.2},
                           {32, 64, 256, false, 1.0, 2.0},   {64, 64, 256, false, 1.0, 3.4},  {64, 128, 512, false, 1.5, 3.4},
                           {128, 128, 512, false, 2.5, 5.6}, {128, 128, 512, true, 2.0, 6.0}, {256, 256, 512, false, 14.0, 15.7}};

int pick_tile(const GemmArgs &g) {
  // (the stride of a single row leads nowhere)
  if ((g.m > 1 && g.lda > kTileStride) || (g.n > 1 && g.ldw > kTileStride)) return 0;
  int best = 0;
  double least = __builtin_inf();
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const Tile &t = kTiles[i];
    const int64_t tiles = cdiv(g.n, t.bn) * cdiv(g.m, t.bm);
    if (t.many && tiles <= kCus) continue;
    if (tiles * t.threads >= (int64_t)1 << 32) continue;  // a grid has fewer threads than that
    if (t.bm > 32 && t.bm >= 2 * g.m) continue;  // half empty: a smaller one does the same
    const double per_k = t.per_k + (i == 0 ? 0.03 * std::min(g.m, 16) : 0.0);
    const double cost = (double)cdiv(tiles, kCus) * (t.fixed * 1e3 + per_k * g.k);
    if (cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

template <typename E>
void launch(const GemmArgs &g, hipStream_t st) {
  switch (pick_tile(g)) {
    case 0: launch_rows<E>(g, st); break;
    case 1: launch_tile<E, 32, 32, 1, 1, 4, 256, 4, 2>(g, st); break;
    case 2: launch_tile<E, 64, 32, 2, 1, 2, 256, 3, 4>(g, st); break;
    case 3: launch_tile<E, 32, 64, 1, 2, 2, 256, 4, 4>(g, st); break;
    case 4: launch_tile<E, 64, 64, 2, 2, 1, 128, 4, 4>(g, st); break;
    case 5: launch_tile<E, 64, 128, 2, 4, 1, 128, 4, 4>(g, st); break;
    case 6: launch_tile<E, 128, 128, 2, 4, 1, 128, 4, 2>(g, st); break;
    case 7: launch_tile<E, 128, 128, 2, 4, 1, 128, 2, 2>(g, st); break;
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
