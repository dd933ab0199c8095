// int8.hpp -- matrices held in 8-bit integers with a scale for each row
// (include/sgemm_int8.h): device helpers and host-side launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
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

// Rows spread thin over groups, in few work-groups (16 columns each; the host
// counts a row of tiles for each group that can have rows).  With the cast first: 8
// groups, 16 rows by 4096 x 4096 26 us (tiles of 64 x 64 35), 16 groups, 24 rows by 2048 x
// 2048 14.7 (15.7); 8 groups, 64 rows by 4096 x 4096 41 (40), 64 groups, 512 rows by 1024
// x 1024 27 (19).
inline bool int8_spread_thin(const Int8Args &p, int cus) {
  const long groups = p.groups < p.M ? p.groups : p.M;
  return p.M <= 2L * p.groups && groups * ((p.N + 15L) / 16) <= 8L * cus;
}

// Up to 16 rows, and rows spread thin over groups, the kernel for few rows, but from 5
// rows on tiles of 64 x 64 where they reach most of the compute units: 16 x 8192 x 8192
// 22.9 us with it (tiles 24), 16 x 8192 x 2048 11.2 (12.3), 16 x 14336 x 4096 23.0 (16.3); 4 x 14336 x
// 4096 19.2 (16.3, but 4 x 8192 x 8192 18.7, 24); 32 x 8192 x 8192 in two blocks of 16
// rows 29.7 (24).
inline bool int8_few_rows(const Int8Args &p, int cus) {
  if (p.offsets) return int8_spread_thin(p, cus);
  return p.M <= 4 || (p.M <= 16 && 4L * ((p.N + 63L) / 64) < 3L * cus);
}

// The tile by times in microseconds: rounds of tiles on the compute units, each with nk
// slices of 128 k.  Groups count with their mean length: the host does not know more.
// Measured on 256 compute units, A cast first (5 to 8 us of it) and C of bfloat16, tiles
// of 64 x 64 / 128 x 128 / 128 x 256 / 256 x 256:
//   N = K = 8192   M = 64   26 / 36 / 55 / 88     M = 256  43 / 45 / 61 / 98
//                  M = 512  76 / 49 / 63 / 101    M = 1024 136 / 91 / 75 / 106
//                  M = 2048 258 / 174 / 143 / 128
//   8192 x 2048    M = 128  13 / 16 / 20 / 30     M = 1024 39 / 32 / 29 / 34
// Stages of a 64 x 64 tile, 2 / 3 / 4: 64 x 8192 x 8192 49 / - / 26 us (two sets of waves
// over k 37, four 32); in groups, where many tiles share a compute unit, 32 groups,
// 48 rows by 4096 x 2048 48 / 43 / 44, 32 groups, 600 rows by 2048 x 2048 45 / 38 / 40, 64
// groups, 512 rows by 1024 x 1024 19.0 / 21.6 / 20.9.  In groups, 64 x 64 and 128 x 128:
// 64 groups, 4099 rows by 1000 x 777 29 and 36, 8 groups, 2000 rows by 4096 x 1024 30 and
// 35, 16 groups, 8192 rows by 2048 x 2048 93 and 80.
enum class Int8Tile { k64_2, k64_3, k64_4, k128, k128x256, k256 };  // 64 x 64: _stages
inline Int8Tile int8_tile(const Int8Args &p, int cus) {
  const long groups = !p.offsets ? 1 : p.groups < p.M ? p.groups : p.M;
  const double mean = (double)p.M / groups, nk = (p.K + 127) / 128;
  auto rounds = [&](long bm, long bn) {
    const double rows = p.offsets ? fmax(1.0, mean / bm + 0.5) : ceil(mean / bm);
    return ceil(groups * rows * ((p.N + bn - 1) / bn) / cus);
  };
  const double c64 = rounds(64, 64) * (0.22 * nk + 1.5) + 6;
  const double c128 = rounds(128, 128) * (0.6 * nk + 2.5) + 6;
  const double c128x256 = rounds(128, 256) * (nk + 3.5) + 6;
  const double c256 = rounds(256, 256) * (1.55 * nk + 5) + 12;
  const double large = fmin(c128x256, c256);
  // Groups of unequal length leave larger tiles emptier.
  if (p.offsets ? mean <= 96 || c64 <= 1.3 * fmin(c128, large) : c64 <= fmin(c128, large))
    return !p.offsets ? Int8Tile::k64_4 : nk <= 8 ? Int8Tile::k64_2 : Int8Tile::k64_3;
  if (c128 <= large) return Int8Tile::k128;
  return c128x256 <= c256 ? Int8Tile::k128x256 : Int8Tile::k256;
}

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
