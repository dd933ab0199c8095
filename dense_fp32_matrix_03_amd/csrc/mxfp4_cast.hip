// mxfp4_cast.hip -- the cast of matrices to microscaled 4-bit floating point
// and back (include/sgemm_mxfp4.h).
//
// Bound by memory: a cast reads 4 (or 2) bytes a value and writes 17/32.
// Every value is read once, by a lane that keeps it until the block's scale
// is known.
//
// k along the stored rows' columns (not transposed): a lane has 8 consecutive
// k, so 4 lanes have a block and 16 a granule of 128 k; the block's largest
// magnitude is found by two exchanges inside a quad of lanes, and the four
// scales of a granule are gathered into the dword that is stored.  Values
// stored transposed: a lane has one row's block, 32 loads that 64 lanes make
// of consecutive addresses, and its largest magnitude needs no exchange; the
// four waves of a work-group have the four blocks of a granule.
#include "mxfp4.hpp"

namespace sgemm {

namespace {

constexpr int kGranule = 128;
constexpr int kRowsPerGroup = 32;  // rows of a work-group, not transposed

// One granule of 32 rows per work-group of 4 waves: 16 lanes a row.  8192 x
// 8192: 53 us from single precision (5.7 TB/s), 30 from bfloat16 (5.7).
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_kernel(CastArgs p) {
  const int tid = threadIdx.x;
  const int g = blockIdx.x % p.granules, tile = blockIdx.x / p.granules;
  const int l16 = tid % 16;
  const int k = g * kGranule + l16 * 8;
  const int left = p.K - k;
#pragma unroll
  for (int i = 0; i < kRowsPerGroup / 16; ++i) {
    const int row = tile * kRowsPerGroup + i * 16 + tid / 16;
    const bool in = row < p.rows;
    float v[8];
    const char *x = static_cast<const char *>(p.X) + ((long)row * p.ldx + k) * (BF16 ? 2 : 4);
    load8<BF16, true>(x, in ? left : 0, v);
    unsigned all;
    const unsigned codes = mxfp4_cast8(v, tid, all);
    if (in) {
      reinterpret_cast<unsigned *>(p.codes)[(long)row * (p.granules * 16) + g * 16 + l16] = codes;
      if (l16 == 0) p.scales[(long)g * p.lds + row] = all;
    }
  }
}

// 64 rows and a granule per work-group; wave w has block w.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_transposed_kernel(CastArgs p) {
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  const int g = blockIdx.x % p.granules, tile = blockIdx.x / p.granules;
  const int row = tile * kWave + lane;
  const int k0 = g * kGranule + w * 32;
  const bool in = row < p.rows;
  // Every lane loads, from the nearest element there is, so that the loads go
  // out together; what lies past K is then dropped.
  const int last = p.K - 1, col = min(row, p.rows - 1);
  float v[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const long at = (long)min(k0 + e, last) * p.ldx + col;
    if constexpr (BF16)
      v[e] = __uint_as_float((unsigned)static_cast<const unsigned short *>(p.X)[at] << 16);
    else
      v[e] = static_cast<const float *>(p.X)[at];
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = k0 + e < p.K ? v[e] : 0.f;
  unsigned top = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) top = max(top, magnitude_bits(v + 8 * q));
  const unsigned s = mxfp4_scale(top);
  __shared__ unsigned char scale[kWave][4];
  scale[lane][w] = (unsigned char)s;
  if (in) {
    uint4 c;
    c.x = mxfp4_codes8(v, s);
    c.y = mxfp4_codes8(v + 8, s);
    c.z = mxfp4_codes8(v + 16, s);
    c.w = mxfp4_codes8(v + 24, s);
    reinterpret_cast<uint4 *>(p.codes)[(long)row * (p.granules * 4) + g * 4 + w] = c;
  }
  __syncthreads();
  if (w == 0 && in)
    p.scales[(long)g * p.lds + row] = *reinterpret_cast<const unsigned *>(scale[lane]);
}

// The scale 2^(s - 127): 2^-127 is below the normal range; 255 is a NaN.
__device__ __forceinline__ float scale_value(unsigned s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (s ? s << 23 : 0x00400000u));
}

// The first N (at most 8) values of a dword of codes.
template <int N = 8>
__device__ __forceinline__ void decode(unsigned codes, float scale, float v[N]) {
  constexpr unsigned kGrid = 0xc8643210u;  // twice the magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const unsigned c = codes >> (4 * e) & 15u;
    const float m = 0.5f * (float)(kGrid >> (4 * (c & 7u)) & 15u);
    v[e] = (c & 8u ? -m : m) * scale;
  }
}

// Exact: a value of the format has at most 2 significant bits.
__device__ __forceinline__ unsigned short to_bf16(float x) {
  return __builtin_bit_cast(unsigned short, (__bf16)x);
}

// The first n (at most 16 bytes) of a lane's values to consecutive elements.
__device__ __forceinline__ void store(unsigned short *x, int n, const float v[8]) {
  if (n >= 8) {
    u32x4_any t;
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = to_bf16(v[2 * e]) | (unsigned)to_bf16(v[2 * e + 1]) << 16;
    __builtin_nontemporal_store(t, reinterpret_cast<u32x4_any *>(x));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) x[e] = to_bf16(v[e]);
  }
}
__device__ __forceinline__ void store(float *x, int n, const float v[4]) {
  if (n >= 4) {
    const f32x4_any t = {v[0], v[1], v[2], v[3]};
    __builtin_nontemporal_store(t, reinterpret_cast<f32x4_any *>(x));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) x[e] = v[e];
  }
}

// A granule of 32 rows per work-group; a lane writes 16 bytes, so that a wave's
// store is of whole rows of the granule.  8192 x 8192: 30 us to bfloat16 (5.6
// TB/s), 51 to single precision (5.9); 80 with eight floats a lane in two stores.
template <bool BF16>
__global__ void __launch_bounds__(256) dequantize_kernel(CastArgs p) {
  using T = std::conditional_t<BF16, unsigned short, float>;
  using Codes = std::conditional_t<BF16, unsigned, unsigned short>;
  constexpr int V = 16 / sizeof(T), kLanes = kGranule / V, kPass = 256 / kLanes;
  const int g = blockIdx.x % p.granules, tile = blockIdx.x / p.granules;
  const int l = threadIdx.x % kLanes;
  const int k = g * kGranule + l * V;
#pragma unroll
  for (int i = 0; i < kRowsPerGroup / kPass; ++i) {
    const int row = tile * kRowsPerGroup + i * kPass + threadIdx.x / kLanes;
    if (row >= p.rows) break;
    const unsigned codes =
        static_cast<const Codes *>(p.codes)[((long)row * p.granules + g) * kLanes + l];
    const unsigned s = p.scales[(long)g * p.lds + row] >> (8 * (l * V / 32)) & 255u;
    float v[V];
    decode<V>(codes, scale_value(s), v);
    store(static_cast<T *>(const_cast<void *>(p.X)) + (long)row * p.ldx + k, p.K - k, v);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) dequantize_transposed_kernel(CastArgs p) {
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  const int g = blockIdx.x % p.granules, tile = blockIdx.x / p.granules;
  const int row = tile * kWave + lane;
  const int k0 = g * kGranule + w * 32;
  if (row >= p.rows) return;
  const uint4 c = reinterpret_cast<const uint4 *>(p.codes)[(long)row * (p.granules * 4) + g * 4 + w];
  const float scale = scale_value(p.scales[(long)g * p.lds + row] >> (8 * w) & 255u);
  float v[32];
  decode(c.x, scale, v);
  decode(c.y, scale, v + 8);
  decode(c.z, scale, v + 16);
  decode(c.w, scale, v + 24);
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    if (k0 + e >= p.K) break;
    const long at = (long)(k0 + e) * p.ldx + row;
    if constexpr (BF16)
      static_cast<unsigned short *>(const_cast<void *>(p.X))[at] = to_bf16(v[e]);
    else
      static_cast<float *>(const_cast<void *>(p.X))[at] = v[e];
  }
}

}  // namespace

hipError_t launch_mxfp4_quantize(bool trans, bool bf16, const CastArgs &p, hipStream_t s) {
  const long tiles = (p.rows + (trans ? kWave : kRowsPerGroup) - 1L) / (trans ? kWave : kRowsPerGroup);
  const dim3 grid((unsigned)(tiles * p.granules)), block(256);
  if (trans && bf16)
    hipLaunchKernelGGL(quantize_transposed_kernel<true>, grid, block, 0, s, p);
  else if (trans)
    hipLaunchKernelGGL(quantize_transposed_kernel<false>, grid, block, 0, s, p);
  else if (bf16)
    hipLaunchKernelGGL(quantize_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(quantize_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(bool trans, bool bf16, const CastArgs &p, hipStream_t s) {
  const long tiles = (p.rows + (trans ? kWave : kRowsPerGroup) - 1L) / (trans ? kWave : kRowsPerGroup);
  const dim3 grid((unsigned)(tiles * p.granules)), block(256);
  if (trans && bf16)
    hipLaunchKernelGGL(dequantize_transposed_kernel<true>, grid, block, 0, s, p);
  else if (trans)
    hipLaunchKernelGGL(dequantize_transposed_kernel<false>, grid, block, 0, s, p);
  else if (bf16)
    hipLaunchKernelGGL(dequantize_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(dequantize_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace sgemm
