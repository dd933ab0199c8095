// piece.hpp -- 16 bytes of a row of single-precision or bfloat16 values.
#pragma once

#include <type_traits>

#include "mxfp4.hpp"  // u32x4_any, f32x4_any

namespace sgemm {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// 16 bytes of a row, at any element: V values, zeros and no access past the n-th.  The
// values are unpacked when they are used, so that several loads go out together.
template <bool BF16>
struct Piece {
  static constexpr int V = BF16 ? 8 : 4;
  using T = std::conditional_t<BF16, unsigned short, float>;
  using Raw = std::conditional_t<BF16, u32x4_any, f32x4_any>;
  Raw raw;
  // whole (the same in all lanes): n >= V for certain, and nothing is tested.
  __device__ __forceinline__ void load(const void *row, long at, int n, bool whole) {
    const T *x = static_cast<const T *>(row) + at;
    if (whole || n >= V) {
      raw = *reinterpret_cast<const Raw *>(x);
    } else if (n > 0) {
      T v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = e < n ? x[e] : T(0);
      __builtin_memcpy(&raw, v, 16);
    } else {
      raw = Raw{0, 0, 0, 0};
    }
  }
  __device__ __forceinline__ void store(void *row, long at, int n) const {
    T *x = static_cast<T *>(row) + at;
    if (n >= V) {
      *reinterpret_cast<Raw *>(x) = raw;
    } else {
      T v[V];
      __builtin_memcpy(v, &raw, 16);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) x[e] = v[e];
    }
  }
  __device__ __forceinline__ void get(float v[V]) const {
    if constexpr (BF16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(raw[e] << 16);
        v[2 * e + 1] = __uint_as_float(raw[e] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = raw[e];
    }
  }
  // The largest magnitude's bits, as those of a float.
  __device__ __forceinline__ unsigned top() const {
    if constexpr (BF16) {
      u16x2 m = {0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, raw[e] & 0x7fff7fffu));
      return (unsigned)max(m[0], m[1]) << 16;
    } else {
      unsigned m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(raw[e]) & 0x7fffffffu);
      return m;
    }
  }
  __device__ __forceinline__ void set(const float v[V]) {
    if constexpr (BF16) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        raw[e] = __builtin_bit_cast(unsigned short, (__bf16)v[2 * e]) |
                 (unsigned)__builtin_bit_cast(unsigned short, (__bf16)v[2 * e + 1]) << 16;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[e] = v[e];
    }
  }
};

}  // namespace sgemm
