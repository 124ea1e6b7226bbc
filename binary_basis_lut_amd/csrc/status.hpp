// status.hpp -- what the host side of every translation unit shares: the status
// helpers (the thread-local message of fluxbin_last_error lives in
// fluxbin.hip) and two small functions on addresses and sizes.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fluxbin.h"

namespace fluxbin {

#define FB_LOCAL __attribute__((visibility("hidden")))
FB_LOCAL fluxbin_status fail(fluxbin_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
FB_LOCAL fluxbin_status hip_fail(hipError_t e, const char *what);
FB_LOCAL fluxbin_status ok();

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace fluxbin
