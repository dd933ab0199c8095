// mxfp4.hpp -- matrices held in microscaled 4-bit floating point
// (include/sgemm_mxfp4.h): device helpers and host-side launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace sgemm {

// A held matrix: codes [rows][Kp / 2], scales [Kp / 128][lds][4].
struct Mxfp4Matrix {
  const unsigned char *codes;
  const unsigned *scales;  // one dword: the four scales of 128 k of a row
  long lds;
};

inline long mxfp4_kp(long K) { return (K + 127) / 128 * 128; }

struct CastArgs {
  int rows, K;
  long ldx;
  int granules;  // Kp / 128
  long lds;
  const void *X;
  void *codes;
  unsigned *scales;
};

hipError_t launch_mxfp4_quantize(bool trans, bool bf16, const CastArgs &p, hipStream_t s);
hipError_t launch_mxfp4_dequantize(bool trans, bool bf16, const CastArgs &p, hipStream_t s);

// C = alpha A B^T + beta C over held B; A held, or values that the kernel casts
// (a.codes points to them and a.lds is their leading dimension).  offsets:
// null, or the groups of sgemm_run_mxfp4_grouped.
struct Mxfp4Args {
  int M, N, K, groups;
  float alpha, beta;
  Mxfp4Matrix a, b;
  void *C;
  long ldc;
  const int64_t *offsets;
};

// Whether the product's kernel is to cast A itself: only then may a_type below
// be other than SGEMM_TYPE_MXFP4.
bool mxfp4_casts(const Mxfp4Args &p, int cus);
// Whether eight waves, not four, share the k of a few rows: from five units of
// 512 k on.  16 x 8192 x 8192 takes 12.3 us with eight and 13.8 with four, 16 x
// 2048 x 2048 3.6 with either.
inline bool mxfp4_eight_sets(long K) { return K > 2048; }
// Picks the kernel for the product.
hipError_t launch_mxfp4_product(const Mxfp4Args &p, int a_type, bool c_bf16, int cus,
                                hipStream_t s);
// mxfp4_tile.hip: tiles through LDS; A held.
hipError_t launch_mxfp4_tile(const Mxfp4Args &p, bool c_bf16, int cus, hipStream_t s);

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Operands in 4 bits fill the lower half of the scaled matrix instructions'
// registers; 4 is the code of the format.
__device__ __forceinline__ i32x8 widen(i32x4 v) {
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
constexpr int kFormatFp4 = 4;

// 16 x 16 x 128 and 32 x 32 x 64 on 4-bit operands, byte S of the scales.
template <int S>
__device__ __forceinline__ f32x4 mfma_fp4_16x16x128(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(a), widen(b), c, kFormatFp4,
                                                          kFormatFp4, S, sa, S, sb);
}
template <int S>
__device__ __forceinline__ f32x16 mfma_fp4_32x32x64(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(a), widen(b), c, kFormatFp4,
                                                         kFormatFp4, S, sa, S, sb);
}

// C[at] = alpha sum + beta C[at], rounded to single precision once after beta C[at]
// and then, for bfloat16, to the nearest.  C is read only when beta != 0.
template <bool CBF16>
__device__ __forceinline__ void store_c(const Mxfp4Args &p, long at, float sum) {
  if constexpr (CBF16) {
    __bf16 *C = static_cast<__bf16 *>(p.C) + at;
    *C = (__bf16)(p.beta == 0.f ? p.alpha * sum : fmaf(p.alpha, sum, p.beta * (float)*C));
  } else {
    float *C = static_cast<float *>(p.C) + at;
    *C = p.beta == 0.f ? p.alpha * sum : fmaf(p.alpha, sum, p.beta * *C);
  }
}

// Four floats (eight bfloat16) at an address aligned to one element.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight consecutive values x[0 .. 7], zeros from the n-th on, as floats.  ONCE:
// nothing else reads them, so 16 bytes of bfloat16 leave the caches alone (8192
// x 8192 30 us for 33; two loads share a line of floats: 57 for 53).
template <bool BF16, bool ONCE = false>
__device__ __forceinline__ void load8(const void *x, int n, float v[8]) {
  if constexpr (BF16) {
    const unsigned short *p = static_cast<const unsigned short *>(x);
    if (n >= 8) {
      const auto *at = reinterpret_cast<const u32x4_any *>(p);
      const u32x4_any t = ONCE ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(t[e] << 16);
        v[2 * e + 1] = __uint_as_float(t[e] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? __uint_as_float((unsigned)p[e] << 16) : 0.f;
    }
  } else {
    const float *p = static_cast<const float *>(x);
    if (n >= 8) {
      const f32x4_any lo = *reinterpret_cast<const f32x4_any *>(p);
      const f32x4_any hi = *reinterpret_cast<const f32x4_any *>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = lo[e];
        v[4 + e] = hi[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.f;
    }
  }
}

// Scale byte of a block whose largest magnitude has the bits `top` (the
// largest of the values' bits without signs: those order as the magnitudes do,
// with infinities and then NaNs at the top).
__device__ __forceinline__ unsigned mxfp4_scale(unsigned top) {
  const unsigned e = top >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// Codes of eight values of a block with scale byte s, the first in the lowest
// four bits.  The values are first multiplied by 2^(127 - s), which is exact
// (the largest ends below 8; what falls below the normal range is far below
// 0.25 and gets code 0 either way); v_cvt_scalef32_pk_fp4_f32 then rounds to
// the nearest value of the format, ties to the even code, at most 6.
__device__ __forceinline__ unsigned mxfp4_codes8(const float v[8], unsigned s) {
  if (s == 255u) return 0u;
  const float up = __uint_as_float((254u - s) << 23);
  unsigned r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * up, v[1] * up, 1.f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * up, v[3] * up, 1.f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * up, v[5] * up, 1.f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * up, v[7] * up, 1.f, 3);
  return r;
}

__device__ __forceinline__ unsigned magnitude_bits(const float v[8]) {
  unsigned top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  return top;
}

// The cast of eight consecutive values, by 16 lanes that together have the 128
// of a granule (lane % 16 its eighth of 16): returns the lane's codes and
// gives every lane the granule's four scale bytes.
__device__ __forceinline__ unsigned mxfp4_cast8(const float v[8], int lane, unsigned &scales) {
  unsigned top = magnitude_bits(v);
  top = max(top, (unsigned)__shfl_xor((int)top, 1));
  top = max(top, (unsigned)__shfl_xor((int)top, 2));
  const unsigned s = mxfp4_scale(top);
  scales = s << (8 * (lane % 16 / 4));
  scales |= (unsigned)__shfl_xor((int)scales, 4);
  scales |= (unsigned)__shfl_xor((int)scales, 8);
  return mxfp4_codes8(v, s);
}

}  // namespace sgemm
