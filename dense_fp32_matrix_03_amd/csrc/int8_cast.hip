// int8_cast.hip -- the cast of matrices to 8-bit integers with a scale for each
// row (include/sgemm_int8.h).
//
// Bound by memory: a cast reads 4 (or 2) bytes a value and writes 1.  8192 x 8192 by graph
// replay: 37 us from bfloat16 (5.5 TB/s), 58 from single precision (5.7); values stored
// transposed 118 and 125, their loads being 2 or 4 bytes a lane and done twice.
#include "int8.hpp"
#include "piece.hpp"

namespace sgemm {

namespace {

// T threads (a wave, or the work-group of four) have a row, 16 bytes each of every 16 T.
// The first 8192 values stay in registers between the search for the largest magnitude
// and the cast (2048 where a wave has the row); longer rows are read again, from the
// caches.
template <bool BF16, int T>
__global__ void __launch_bounds__(256) int8_quantize_kernel(Int8CastArgs p) {
  static_assert(T == 64 || T == 256, "a wave or a work-group has a row");
  using P = Piece<BF16>;
  constexpr int V = P::V, kStep = V * T, kHeld = BF16 ? 4 : 8;
  const int t = threadIdx.x % T;
  const long row = (long)blockIdx.x * (256 / T) + threadIdx.x / T;
  if (T < 256 && row >= p.rows) return;  // whole waves: no barrier follows
  const char *x = static_cast<const char *>(p.X) + row * p.ldx * (BF16 ? 2 : 4);
  P held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    held[i].load(x, i * kStep + t * V, p.K - (i * kStep + t * V), (i + 1) * kStep <= p.K);
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) top = max(top, held[i].top());
  for (int k = kHeld * kStep + t * V; k < p.K; k += kStep) {
    P v;
    v.load(x, k, p.K - k, false);
    top = max(top, v.top());
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) top = max(top, (unsigned)__shfl_xor((int)top, d));
  if constexpr (T == 256) {
    __shared__ unsigned tops[4];
    if (threadIdx.x % kWave == 0) tops[threadIdx.x / kWave] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  }
  const Int8Scale s(int8_scale(top));
  if (t == 0) p.scales[row] = s.scale;
  const int kp = (p.K + 127) / 128 * 128;
  char *codes = p.codes + row * p.ldq;
  auto store = [&](int k, const P &v) {
    if (k >= kp) return;
    float f[V];
    unsigned c[V / 4];
    v.get(f);
    int8_codes<V>(s, f, c);
    __builtin_memcpy(__builtin_assume_aligned(codes + (k / 128) * p.slice + k % 128, V), c, V);
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) store(i * kStep + t * V, held[i]);
  for (int k = kHeld * kStep + t * V; k < kp; k += kStep) {
    P v;
    v.load(x, k, p.K - k, false);
    store(k, v);
  }
}

// Values stored transposed: a work-group has 32 rows (neighbouring columns of X),
// kParts threads each; a thread takes 16 consecutive k of every 16 kParts.  Loads of 32
// lanes adjoin.  Two passes: X is read twice.
constexpr int kParts = 32;

template <bool BF16>
__global__ void __launch_bounds__(32 * kParts) int8_quantize_transposed_kernel(Int8CastArgs p) {
  const int c = threadIdx.x % 32, part = threadIdx.x / 32;
  const long row = (long)blockIdx.x * 32 + c;
  // Every thread loads, from the nearest element there is, so that the loads go
  // out together; what lies past K or the last row is then dropped.
  const long col = min(row, (long)p.rows - 1);
  auto load = [&](int k0, float v[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const long at = (long)min(k0 + e, p.K - 1) * p.ldx + col;
      if constexpr (BF16)
        v[e] = __uint_as_float((unsigned)static_cast<const unsigned short *>(p.X)[at] << 16);
      else
        v[e] = static_cast<const float *>(p.X)[at];
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = k0 + e < p.K ? v[e] : 0.f;
  };
  unsigned top = 0;
  for (int k = part * 16; k < p.K; k += 16 * kParts) {
    float v[16];
    load(k, v);
    top = max(top, max(magnitude_bits(v), magnitude_bits(v + 8)));
  }
  __shared__ unsigned tops[kParts][32];
  tops[part][c] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kParts; ++i) top = max(top, tops[i][c]);
  if (row >= p.rows) return;
  const Int8Scale s(int8_scale(top));
  if (part == 0) p.scales[row] = s.scale;
  const int kp = (p.K + 127) / 128 * 128;
  for (int k = part * 16; k < kp; k += 16 * kParts) {
    float v[16];
    load(k, v);
    unsigned c[4];
    int8_codes<16>(s, v, c);
    *reinterpret_cast<uint4 *>(p.codes + row * p.ldq + (k / 128) * p.slice + k % 128) =
        uint4{c[0], c[1], c[2], c[3]};
  }
}

}  // namespace

hipError_t launch_int8_quantize(bool trans, bool bf16, const Int8CastArgs &p, hipStream_t s) {
  const dim3 block(256);
  if (trans) {
    const dim3 grid((unsigned)((p.rows + 31L) / 32)), wide(32 * kParts);
    if (bf16)
      hipLaunchKernelGGL(int8_quantize_transposed_kernel<true>, grid, wide, 0, s, p);
    else
      hipLaunchKernelGGL(int8_quantize_transposed_kernel<false>, grid, wide, 0, s, p);
  } else if (p.K > 2048) {
    const dim3 grid((unsigned)p.rows);
    if (bf16)
      hipLaunchKernelGGL((int8_quantize_kernel<true, 256>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((int8_quantize_kernel<false, 256>), grid, block, 0, s, p);
  } else {
    const dim3 grid((unsigned)((p.rows + 3L) / 4));
    if (bf16)
      hipLaunchKernelGGL((int8_quantize_kernel<true, 64>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((int8_quantize_kernel<false, 64>), grid, block, 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace sgemm
