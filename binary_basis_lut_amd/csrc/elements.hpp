// elements.hpp -- activation elements of the 8-bit operators: fp16, bf16 and
// fp32 values, converted to and from fp32, moved eight at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fluxbin {

// A unit is eight consecutive elements, held as they are stored.  Global memory
// takes a 16-byte access at any element's address (gfx950 runs in the unaligned
// access mode on Linux), so rows of odd length and odd strides move at full
// width too; the vector types say what alignment the compiler may assume.
constexpr int kUnit = 8;

typedef uint32_t words4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t words2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t bytes8 __attribute__((ext_vector_type(2), aligned(1)));
typedef float floats4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename E>
struct HalfUnit {  // fp16 and bf16
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const { return E::load((uint16_t)(w[i / 2] >> (16 * (i % 2)))); }
  __device__ __forceinline__ void set(const float (&f)[kUnit]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)E::round(f[2 * i]) | (uint32_t)E::round(f[2 * i + 1]) << 16;
  }
  __device__ __forceinline__ void fill(uint16_t v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v | (uint32_t)v << 16;
  }
  __device__ __forceinline__ void read(const uint16_t *p) {
    const words4 v = *reinterpret_cast<const words4 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  }
  __device__ __forceinline__ void write(uint16_t *p) const {
    words4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
    *reinterpret_cast<words4 *>(p) = v;
  }
  __device__ __forceinline__ void put(int i, uint16_t v) {
    w[i / 2] = i % 2 ? (w[i / 2] & 0xffffu) | (uint32_t)v << 16 : (w[i / 2] & 0xffff0000u) | v;
  }
  __device__ __forceinline__ uint16_t at(int i) const { return (uint16_t)(w[i / 2] >> (16 * (i % 2))); }
};

struct F16 {
  typedef uint16_t raw;
  typedef HalfUnit<F16> unit;
  static __device__ __forceinline__ float load(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ raw round(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};

struct BF16 {
  typedef uint16_t raw;
  typedef HalfUnit<BF16> unit;
  static __device__ __forceinline__ float load(raw v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ raw round(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};

struct FloatUnit {
  float f[kUnit];
  __device__ __forceinline__ float get(int i) const { return f[i]; }
  __device__ __forceinline__ void set(const float (&v)[kUnit]) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = v[i];
  }
  __device__ __forceinline__ void fill(float v) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = v;
  }
  __device__ __forceinline__ void read(const float *p) {
    const floats4 a = *reinterpret_cast<const floats4 *>(p), b = *reinterpret_cast<const floats4 *>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
  __device__ __forceinline__ void write(float *p) const {
    *reinterpret_cast<floats4 *>(p) = floats4{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<floats4 *>(p + 4) = floats4{f[4], f[5], f[6], f[7]};
  }
  __device__ __forceinline__ void put(int i, float v) { f[i] = v; }
  __device__ __forceinline__ float at(int i) const { return f[i]; }
};

struct F32 {
  typedef float raw;
  typedef FloatUnit unit;
  static __device__ __forceinline__ float load(raw v) { return v; }
  static __device__ __forceinline__ raw round(float f) { return f; }
};

// The elements [at, at + 8) of a row of n: a whole unit, or the row's last
// elements one by one with `fill` behind them (a fill for at >= n, too).
template <typename E>
__device__ __forceinline__ typename E::unit load_part(const typename E::raw *row, int64_t at, int64_t n, float fill) {
  typename E::unit u;
  if (at + kUnit <= n) {
    u.read(row + at);
  } else {
    u.fill(E::round(fill));
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if (at + i < n) u.put(i, row[at + i]);
  }
  return u;
}
template <typename E>
__device__ __forceinline__ void store_part(typename E::raw *row, int64_t at, int64_t n, const typename E::unit &u) {
  if (at + kUnit <= n) {
    u.write(row + at);
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if (at + i < n) row[at + i] = u.at(i);
  }
}

}  // namespace fluxbin
