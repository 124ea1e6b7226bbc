// lds_loads.hpp -- loads from global memory straight into LDS, and the waits that
// go with them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fluxbin {

#define FB_LDS __attribute__((address_space(3)))
#define FB_GLB __attribute__((address_space(1)))

// The same address, known to be the same in every lane: a buffer descriptor in
// vector registers would be read out lane by lane around every load.
__device__ __forceinline__ const int8_t *in_scalars(const int8_t *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const int8_t *>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                                          (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
// A buffer of `bytes` 0 gives zeros and touches no memory.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, bytes, 0x00027000);
}
// Sixteen bytes per lane from global memory straight into LDS: lane l's piece, at
// base + soff + voff, lands at dst + 16 l.  A buffer load rather than a global
// one: the compiler takes a direct global load for an LDS access too and would
// then wait for all fragment reads in flight wherever it waits for some.  ONCE: of
// data that nobody reads again, which then does not push other data out of the L2.
template <bool ONCE = false>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t base, uint32_t voff, uint32_t soff, FB_LDS int8_t *dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (FB_LDS void *)dst, 16, voff, soff, 0, ONCE ? 2 : 0);
}

// Waits until at most `vm` of the wave's vector-memory operations and none of
// its LDS operations are outstanding, then for the workgroup.
template <int VM>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(VM < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | (VM >> 4) << 14);  // lgkmcnt 0, expcnt any
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The same without a meeting, for waves that share nothing: until at most VM
// vector-memory operations are outstanding, and until no LDS operation is.
template <int VM>
__device__ __forceinline__ void wait_for_loads() {
  static_assert(VM < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | 15 << 8 | (VM >> 4) << 14);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_for_reads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | 7 << 4 | 3 << 14);  // lgkmcnt 0, the others any
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace fluxbin
