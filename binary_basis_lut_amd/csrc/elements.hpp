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
  // Element j of N units, for a j that differs between lanes.
  template <int N>
  static __device__ __forceinline__ float pick(const HalfUnit (&u)[N], int j) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) v = j / 2 == i ? u[i / 4].w[i % 4] : v;
    return E::load((uint16_t)(v >> (16 * (j % 2))));
  }
  // Drops the first n elements (0 .. 7) and fills up behind the rest.
  __device__ __forceinline__ void drop(int n, uint16_t v) {
    const uint32_t f = v | (uint32_t)v << 16;
    if (n & 4) {
      w[0] = w[2];
      w[1] = w[3];
      w[2] = w[3] = f;
    }
    if (n & 2) {
      w[0] = w[1];
      w[1] = w[2];
      w[2] = w[3];
      w[3] = f;
    }
    if (n & 1) {
      w[0] = w[0] >> 16 | w[1] << 16;
      w[1] = w[1] >> 16 | w[2] << 16;
      w[2] = w[2] >> 16 | w[3] << 16;
      w[3] = w[3] >> 16 | f << 16;
    }
  }
  __device__ __forceinline__ uint16_t at(int i) const { return (uint16_t)(w[i / 2] >> (16 * (i % 2))); }
  // Keeps the unit as it is stored across this point: without it the compiler
  // carries the converted values, twice the registers.
  __device__ __forceinline__ void hold() { asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3])); }
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
  template <int N>
  static __device__ __forceinline__ float pick(const FloatUnit (&u)[N], int j) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnit * N; ++i) v = j == i ? u[i / kUnit].f[i % kUnit] : v;
    return v;
  }
  __device__ __forceinline__ void drop(int n, float v) {
#pragma unroll
    for (int s = 4; s > 0; s /= 2)
      if (n & s) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) f[i] = i + s < kUnit ? f[i + s] : v;
      }
  }
  __device__ __forceinline__ float at(int i) const { return f[i]; }
  __device__ __forceinline__ void hold() {}
};

struct F32 {
  typedef float raw;
  typedef FloatUnit unit;
  static __device__ __forceinline__ float load(raw v) { return v; }
  static __device__ __forceinline__ raw round(float f) { return f; }
};

// The elements [at, at + 8) of a row of n, with `fill` for those at n and
// beyond, in two steps so that the first steps of several units are in flight
// together: a row's last, incomplete unit is read eight elements from the
// row's end and then moved into place.  Rows of less than eight elements (TINY)
// are read one by one.  I is int for rows whose positions fit it (the row's
// address then stays in scalar registers), else int64_t.
template <typename E, bool TINY, typename I>
__device__ __forceinline__ typename E::unit load_part(const typename E::raw *row, I at, I n, float fill) {
  typename E::unit u;
  u.fill(E::round(fill));
  if (TINY) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if (at + i < n) u.put(i, row[at + i]);
  } else if (at < n) {
    u.read(row + (at + kUnit <= n ? at : n - kUnit));
  }
  return u;
}
template <typename E, bool TINY, typename I>
__device__ __forceinline__ void settle_part(typename E::unit &u, I at, I n, float fill) {
  if (!TINY && at < n && at + kUnit > n) u.drop((int)(at + kUnit - n), E::round(fill));
}
template <typename E, typename I>
__device__ __forceinline__ void store_part(typename E::raw *row, I at, I n, const typename E::unit &u) {
  if (at + kUnit <= n) {
    u.write(row + at);
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if (at + i < n) row[at + i] = u.at(i);
  }
}

}  // namespace fluxbin
