// key_weight.hpp -- what one key weighs in a row that is computed key by key.  Plain
// enough for the host's compiler too, so that it can be tried there over all of fp32.
#pragma once

#include <math.h>

namespace fluxbin {

#if defined(__HIP__)
#define FB_BOTH __host__ __device__ __forceinline__
#else
#define FB_BOTH inline
#endif

constexpr float kWeightShift = 7.0f;

FB_BOTH float power_of_two(float x) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_exp2f(x);
#else
  return exp2f(x);
#endif
}

// The weight of a key of score s under the maximum m.  The difference comes before the
// product: c s and c m may both pass fp32's range.  A key that is not there weighs
// nothing whatever s and m are.
FB_BOTH float key_weight(bool there, float s, float m, float c) {
  return there ? power_of_two(fmaf(s - m, c, kWeightShift)) : 0.0f;
}

}  // namespace fluxbin
