// status.hpp -- what the host side of every translation unit shares: the status
// helpers (the thread-local message of fluxbin_last_error lives in
// fluxbin.hip) and small functions on addresses and sizes.
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

// Whether one of `rows` rows of `elems` elements, `ldp` apart from p on, meets one of as
// many rows `ldq` apart from q on (strides of at least `elems`).  Rows of one buffer's
// columns lie between each other and do not.
inline bool rows_overlap(const void *p, int64_t ldp, const void *q, int64_t ldq, int64_t rows, int64_t elems, int bytes) {
  typedef __int128 wide;
  const wide x = (wide)reinterpret_cast<uintptr_t>(p), y = (wide)reinterpret_cast<uintptr_t>(q), sp = (wide)ldp * bytes,
             sq = (wide)ldq * bytes, width = (wide)elems * bytes;
  if (y >= x + (rows - 1) * sp + width || x >= y + (rows - 1) * sq + width) return false;
  // row j of q lies `rest` behind the beginning of row i of p: does it meet that or the next one?
  const auto meets = [&](wide at, wide most_i, wide least_i) {
    wide i = at / sp, rest = at % sp;
    if (rest < 0) --i, rest += sp;
    return (rest < width && i >= least_i && i <= most_i) || (sp - rest < width && i + 1 >= least_i && i + 1 <= most_i);
  };
  if (ldp == ldq) return meets(y - x, rows - 1, 1 - rows);  // i - j, which any two rows may have
  for (int64_t j = 0; j < rows; ++j)
    if (meets(y - x + j * sq, rows - 1, 0)) return true;
  return false;
}

}  // namespace fluxbin
