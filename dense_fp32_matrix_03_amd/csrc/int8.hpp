// int8.hpp -- matrices held in 8-bit integers with a scale for each row
// (include/sgemm_int8.h): device helpers and host-side launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "mxfp4.hpp"  // load8: eight values of either type
#include "slice_tile.hpp"

namespace sgemm {

inline long int8_kp(long K) { return (K + 127) / 128 * 128; }

struct Int8CastArgs {
  int rows, K;
  long ldx;
  const void *X;
  char *codes;
  long ldq, slice;  // as in Int8Matrix
  float *scales;
};

hipError_t launch_int8_quantize(bool trans, bool bf16, const Int8CastArgs &p, hipStream_t s);

// A held matrix: slices of 128 k of a row lie `slice` bytes apart, rows of a slice
// `ld`: 128 and the user's ldq, or in the workspace 128 * rows and 128 (the
// reason stands at SliceRows in slice_tile.hpp).
struct Int8Matrix {
  const char *codes;
  const float *scales;
  long ld;
  long slice;
  __device__ __forceinline__ SliceRows tile_rows(long first, int rows) const {
    return {codes + first * ld, (int)ld, slice, rows};
  }
};

// C = alpha A B^T + beta C over held operands; or A of values that the kernel
// casts (a.codes points to them and a.ld is their leading dimension).  offsets:
// null, or the groups of sgemm_run_int8_grouped.
struct Int8Args {
  int M, N, K, groups;
  float alpha, beta;
  Int8Matrix a, b;
  void *C;
  long ldc;
  const int64_t *offsets;
};

// Whether the product's kernel is to cast A itself: only then may a_type below
// be other than SGEMM_TYPE_INT8.
bool int8_casts(const Int8Args &p, int cus);
// Picks the kernel for the product.
hipError_t launch_int8_product(const Int8Args &p, int a_type, bool c_bf16, int cus, hipStream_t s);
// int8_tile.hip: tiles through LDS; A held.
hipError_t launch_int8_tile(const Int8Args &p, bool c_bf16, int cus, hipStream_t s);

typedef int i32x16 __attribute__((ext_vector_type(16)));

// The scale of a row whose largest magnitude has the bits `top`: NaN where that
// is an infinity or a NaN.  The division is the correctly rounded one.
__device__ __forceinline__ float int8_scale(unsigned top) {
  return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
}

// What a row's casts share: the scale, and an estimate of its reciprocal.  Codes
// are 0 where the scale is 0 or NaN.
struct Int8Scale {
  float scale, inverse;
  bool zero;
  __device__ __forceinline__ explicit Int8Scale(float s) : Int8Scale(s, 1.0f / s) {}
  __device__ __forceinline__ Int8Scale(float s, float i) : scale(s), inverse(i), zero(!(s > 0.f)) {}
  // The whole number nearest to x / scale, halves to the even one.  x times the
  // reciprocal is off by at most 127 2 2^-24, so q is the nearest or, next
  // to a half, the other one; x - q scale is exact (a multiple of the smaller of
  // the two's units, below scale in magnitude), and says which.  Scales so small
  // that the reciprocal overflows are divided by.
  __device__ __forceinline__ int code(float x) const {
    if (zero) return 0;
    float q = rintf(inverse <= 3.4028235e38f ? x * inverse : x / scale);
    const float r = fmaf(-q, scale, x), twice = 2.f * fabsf(r);
    const bool odd = ((int)q & 1) != 0;
    if (twice > scale || (twice == scale && odd)) q += r > 0.f ? 1.f : -1.f;
    return (int)fminf(fmaxf(q, -127.f), 127.f);
  }
};

// Four codes as bytes, the first lowest.
__device__ __forceinline__ unsigned int8_pack(int a, int b, int c, int d) {
  return (unsigned)(a & 255) | (unsigned)(b & 255) << 8 | (unsigned)(c & 255) << 16 |
         (unsigned)d << 24;
}

// N values' codes, packed.  A fused multiply-add with 1.5
// 2^23 rounds x times the reciprocal to a whole number, halves to even, and has its
// code in its last bits.  The reciprocal is off by 2^-24 of itself, the product by less
// than 2^-17, so that the code is the right one unless the product is that near to a
// half: then, and for scales that have few bits, each is found as in Int8Scale.
template <int N>
__device__ __forceinline__ void int8_codes(const Int8Scale &s, const float v[N],
                                           unsigned packed[N / 4]) {
  if (s.zero) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) packed[i] = 0;
    return;
  }
  constexpr float kWhole = 12582912.f;
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    unsigned y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[4 * i + e], whole = fmaf(x, s.inverse, kWhole);
      worst = fmaxf(worst, fabsf(fmaf(x, s.inverse, kWhole - whole)));
      y[e] = __float_as_uint(whole);
    }
    // v_perm_b32: bytes 0 .. 3 are the second operand's, 4 .. 7 the first one's.
    packed[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(y[3], y[2], 0x0c0c0400u),
                                      __builtin_amdgcn_perm(y[1], y[0], 0x0c0c0400u), 0x05040100u);
  }
  if (__ballot(!(worst < 0.5f - 0x1p-16f)) != 0 || !(s.scale >= 0x1p-100f)) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      packed[i] = int8_pack(s.code(v[4 * i]), s.code(v[4 * i + 1]), s.code(v[4 * i + 2]),
                            s.code(v[4 * i + 3]));
  }
}

__device__ __forceinline__ float int8_value(int sum, float sa, float sb) {
  return (float)sum * sa * sb;
}

}  // namespace sgemm
