// wave_ops.hpp -- reductions over the 64 lanes of a wave with DPP moves: four
// shifts inside the rows of 16, then the row sums handed on (row_bcast), six
// VALU instructions whose result is in lane 63 and read from there.  The order
// is fixed, so sums repeat bitwise.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fluxbin {

// v moved by one DPP step; lanes without a source (or outside ROWS) get `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_move(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xf, false);
}

// Op::join(a, b) for values made of Op::words 32-bit words; Op::identity() is
// what lanes without a source join.
template <typename Op, int CTRL, int ROWS>
__device__ __forceinline__ typename Op::type reduce_step(typename Op::type v) {
  union U {
    typename Op::type t;
    int w[sizeof(typename Op::type) / 4];
  };
  U from, none, to;
  from.t = v;
  none.t = Op::identity();
#pragma unroll
  for (unsigned i = 0; i < sizeof(typename Op::type) / 4; ++i) to.w[i] = dpp_move<CTRL, ROWS>(none.w[i], from.w[i]);
  return Op::join(v, to.t);
}

template <typename Op>
__device__ __forceinline__ typename Op::type wave_reduce(typename Op::type v) {
  v = reduce_step<Op, 0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v = reduce_step<Op, 0x112, 0xf>(v);
  v = reduce_step<Op, 0x114, 0xf>(v);
  v = reduce_step<Op, 0x118, 0xf>(v);
  v = reduce_step<Op, 0x142, 0xa>(v);  // row_bcast 15 into rows 1 and 3
  v = reduce_step<Op, 0x143, 0xc>(v);  // row_bcast 31 into rows 2 and 3
  union U {
    typename Op::type t;
    int w[sizeof(typename Op::type) / 4];
  };
  U r;
  r.t = v;
#pragma unroll
  for (unsigned i = 0; i < sizeof(typename Op::type) / 4; ++i) r.w[i] = __builtin_amdgcn_readlane(r.w[i], 63);
  return r.t;
}

struct SumF {
  typedef float type;
  static __device__ __forceinline__ float identity() { return 0.0f; }
  static __device__ __forceinline__ float join(float a, float b) { return a + b; }
};
struct MaxF {
  typedef float type;
  static __device__ __forceinline__ float identity() { return -__builtin_inff(); }
  static __device__ __forceinline__ float join(float a, float b) { return fmaxf(a, b); }
};
struct MaxU {
  typedef uint32_t type;
  static __device__ __forceinline__ uint32_t identity() { return 0; }
  static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
};
struct MaxKey {
  typedef uint64_t type;
  static __device__ __forceinline__ uint64_t identity() { return 0; }
  static __device__ __forceinline__ uint64_t join(uint64_t a, uint64_t b) { return a > b ? a : b; }
};

}  // namespace fluxbin
