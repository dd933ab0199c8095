// orthogonalize.hip -- the products of Newton-Schulz steps
// (include/sgemm_orthogonalize.h) on the half-precision matrix cores.
//
// A value v is held as high + low, two half-precision numbers, high = v rounded and
// low = v - high rounded: off by 2^-22 of v at most.  A product a b is then
// al bh + ah bl + ah bh, three instructions instead of one (al bl, below 2^-22 of
// it, is left out).  Every row is scaled by a power of two of its own, which keeps it
// below 2^15 (RowScale).  One power of two for a matrix was up to 1 us a launch
// faster (16 x 256 x 512 125.6 us for 145) and left rows and columns that are small
// against the others with few digits.
//
// With m <= n a step is S = Z Z^T, P = b S + c S S and a Z + P Z.  All three are
// products of rows by rows once Z is held transposed too: the epilogue writes a
// result as it is and transposed, each by its rows' scales.  S and P are symmetric: blocks
// on and below the diagonal are computed, and written to both sides.  All tiles add
// an element's terms in the same order.
//
// Three times the operations of the formula at half precision's rate (1.33 PFLOP/s in a
// large library product) are the floor.  Five steps, microseconds by the card and the floor:
//   1 x 2048 x 4096      978 - 1070  676    the power limit: a Z + P Z 97 (1.06 PFLOP/s), S
//                                           and P 53 (136 tiles on 256 compute units)
//   1 x 1500 x 1001      216 - 256   62     S and P 13 each, a Z + P Z 19: 1.5 rounds of
//                                           tiles, fixed costs of 4 to 5 us a launch
//   16 x 256 x 512       134 - 161   21     17 launches of 5 to 14 us, of which 4 to 6 are
//                                           fixed: first loads from memory, and the stores
// Sizes and the split are bound by memory: 2048 x 4096 11.8 us (2.9 TB/s), 4.7 for the
// parts, and 18 (5.6).
#include <math.h>

#include "orthogonalize.hpp"
#include "piece.hpp"
#include "slice_tile.hpp"

namespace sgemm {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// A slice of 128 bytes a row is 32 k: chunks 0 .. 3 their high pieces, 4 .. 7 the
// low ones; v_mfma_f32_32x32x16_f16 takes 8 of them from each half of the lanes.
struct SplitFormat {
  typedef f32x16 Acc;
  struct Frag {
    f16x8 high, low;
  };
  static constexpr int kSteps = 2, kReads = 2, kMfma = 3, kChains = 1;
  template <int S, class At>
  __device__ __forceinline__ static Frag load(int half, At at) {
    return {__builtin_bit_cast(f16x8, *at(2 * S + half)),
            __builtin_bit_cast(f16x8, *at(4 + 2 * S + half))};
  }
  template <int I>
  __device__ __forceinline__ static void mma(const Frag &a, const Frag &b, Acc &c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(I == 0 ? a.low : a.high, I == 1 ? b.low : b.high, c,
                                               0, 0, 0);
  }
};

__device__ __forceinline__ void split(float v, _Float16 &high, _Float16 &low) {
  high = (_Float16)v;
  low = (_Float16)(v - (float)high);
}

template <bool BF16>
__device__ __forceinline__ float load1(const void *x, long at) {
  if constexpr (BF16)
    return __uint_as_float((unsigned)static_cast<const unsigned short *>(x)[at] << 16);
  else
    return static_cast<const float *>(x)[at];
}

// A wave's LDS accesses keep their order; this keeps the compiler's.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

__device__ __forceinline__ double group_sum(double v) {  // of 256 threads
  __shared__ double part[4];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  return part[0] + part[1] + part[2] + part[3];
}

// Part blockIdx.x of matrix blockIdx.y: a wave has every 4 n_parts-th run of 512
// elements of a row, and loads four of them together.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_norm_kernel(OrthoNormArgs p) {
  using P = Piece<BF16>;
  constexpr int kTogether = 4, kPieces = kNormRun / (kWave * P::V);
  const long base = (long)blockIdx.y * p.strideX;
  const int runs = (p.N + kNormRun - 1) / kNormRun;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const long step = 4 * p.n_parts, all = (long)p.M * runs;
  double sum = 0;
  for (long u0 = blockIdx.x * 4 + wave; u0 < all; u0 += kTogether * step) {
    P x[kTogether][kPieces];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const long u = u0 + i * step, row = u < all ? u / runs : 0;
      const int n0 = u < all ? (int)(u - row * runs) * kNormRun : p.N;
      const bool whole = p.N - n0 >= kNormRun;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int n = n0 + (k * kWave + lane) * P::V;
        x[i][k].load(p.X, base + row * p.ldx + n, p.N - n, whole);
      }
    }
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        float v[P::V];
        x[i][k].get(v);
#pragma unroll
        for (int e = 0; e < P::V; ++e) sum += (double)v[e] * (double)v[e];
      }
  }
  sum = group_sum(sum);
  if (threadIdx.x == 0) p.parts[(long)blockIdx.y * p.n_parts + blockIdx.x] = sum;
}

// A block of 32 rows of 128 bytes in LDS, chunk c of 16 bytes at c ^ (row % 8): a
// wave reads and writes it without bank conflicts both as 64 lanes' 16 bytes in
// their order, as memory has it, and by columns, as the matrix instructions do.
struct BlockImage {
  char *at;
  __device__ __forceinline__ char *chunk(int row, int c) const {
    return at + row * 128 + ((c ^ (row & 7)) << 4);
  }
  // Lane's chunk of the i-th quarter (8 rows).
  __device__ __forceinline__ slice_i32x4 *linear(int lane, int i) const {
    return reinterpret_cast<slice_i32x4 *>(chunk(8 * i + lane / 8, lane % 8));
  }
};

// The largest of a half of the lanes, in its last one, by moves inside rows of 16 and from
// row to row.
__device__ __forceinline__ int half_wave_max(int v) {
  constexpr int least = -(1 << 30);
  v = max(v, __builtin_amdgcn_update_dpp(least, v, 0x111, 0xf, 0xf, false));  // 1 lane before
  v = max(v, __builtin_amdgcn_update_dpp(least, v, 0x112, 0xf, 0xf, false));  // 2
  v = max(v, __builtin_amdgcn_update_dpp(least, v, 0x114, 0xf, 0xf, false));  // 4
  v = max(v, __builtin_amdgcn_update_dpp(least, v, 0x118, 0xf, 0xf, false));  // 8
  return max(v, __builtin_amdgcn_update_dpp(least, v, 0x142, 0xa, 0xf, false));  // the row before's
}

// 2^x.
__device__ __forceinline__ float power_of_two(int x) {
  return __uint_as_float((unsigned)(min(max(x, -126), 127) + 127) << 23);
}

// One of two for each lane, out of scalar registers: a reference to one or the other would
// read the kernel's arguments through memory.
__device__ __forceinline__ RowScale either(bool first, const RowScale a, const RowScale b) {
  return {first ? a.norm : b.norm, first ? a.count : b.count, first ? a.shift : b.shift,
          first ? a.add : b.add, first ? a.cap : b.cap};
}

// The pieces of a block of sums (as the matrix instructions leave them) times `scale` of
// each row to an image of the block.
__device__ __forceinline__ void split_block(const float v[16], const float scale[16], int r32,
                                            int half, const BlockImage &d) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    _Float16 h, l;
    split(v[e] * scale[e], h, l);
    const int m = 8 * (e / 4) + 4 * half + e % 4;
    reinterpret_cast<_Float16 *>(d.chunk(m, r32 / 8))[r32 % 8] = h;
    reinterpret_cast<_Float16 *>(d.chunk(m, 4 + r32 / 8))[r32 % 8] = l;
  }
}
// The same of its transpose, whose row is the lane's.
__device__ __forceinline__ void split_transposed(const float v[16], float scale, int r32, int half,
                                                 const BlockImage &t) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f16x4 high, low;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      _Float16 h, l;
      split(v[4 * q + e] * scale, h, l);
      high[e] = h;
      low[e] = l;
    }
    *reinterpret_cast<f16x4 *>(t.chunk(r32, q) + 8 * half) = high;
    *reinterpret_cast<f16x4 *>(t.chunk(r32, 4 + q) + 8 * half) = low;
  }
}
// The floats: as they are, or transposed.
__device__ __forceinline__ void floats_block(const float v[16], bool turned, int r32, int half,
                                             const BlockImage &d) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int m = 8 * q + 4 * half;
    if (turned) {
      *reinterpret_cast<f32x4 *>(d.chunk(r32, m / 4)) =
          f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<float *>(d.chunk(m + e, r32 / 4))[r32 % 4] = v[4 * q + e];
    }
  }
}

// The rows of an image below `rows` to the matrix's block at (r0, c0).
__device__ __forceinline__ void store_block(const SplitMatrix &x, int batch, int r0, int c0,
                                            int rows, int lane, const BlockImage &image) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = r0 + 8 * k + lane / 8;
    if (r < rows)
      *reinterpret_cast<slice_i32x4 *>(x.place(batch, r, c0) + lane % 8 * 16) =
          *image.linear(lane, k);
  }
}

// A work-group's band of rows by 512 columns: a wave has every fourth row, 8 columns a
// lane, and loads four of its rows together.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_sizes_kernel(OrthoSizesArgs p) {
  using P = Piece<BF16>;
  constexpr int kTogether = 4, kPieces = kNormRun / (kWave * P::V);
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int run = blockIdx.x % p.runs, band = blockIdx.x / p.runs;
  const long batch = blockIdx.y;
  const int n0 = run * kNormRun, end = min((band + 1) * p.band, p.M);
  const bool whole = p.N - n0 >= kNormRun;
  const long base = batch * p.strideX;
  unsigned *const row_parts = p.row_parts + (batch * p.runs + run) * p.M;
  double sum = 0;
  unsigned top[kPieces][P::V];  // of the lane's columns
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
#pragma unroll
    for (int e = 0; e < P::V; ++e) top[k][e] = 0;
  for (int row = band * p.band + wave; row < end; row += 4 * kTogether) {
    P x[kTogether][kPieces];
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int n = n0 + (k * kWave + lane) * P::V, r = row + 4 * i;
        x[i][k].load(p.X, base + min(r, end - 1) * p.ldx + n, r < end ? p.N - n : 0,
                     whole && r < end);
      }
    unsigned most[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      most[i] = 0;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        float v[P::V];
        x[i][k].get(v);
        most[i] = max(most[i], x[i][k].top());
#pragma unroll
        for (int e = 0; e < P::V; ++e) {
          sum += (double)v[e] * (double)v[e];
          top[k][e] = max(top[k][e], __float_as_uint(v[e]) & 0x7fffffffu);
        }
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
#pragma unroll
      for (int i = 0; i < kTogether; ++i)
        most[i] = max(most[i], (unsigned)__shfl_xor((int)most[i], d));
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
      if (lane == 0 && row + 4 * i < end) row_parts[row + 4 * i] = most[i];
  }
  __shared__ unsigned tops[4][kNormRun];
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
#pragma unroll
    for (int e = 0; e < P::V; ++e) tops[wave][(k * kWave + lane) * P::V + e] = top[k][e];
  sum = group_sum(sum);  // its barrier is for tops too
  if (threadIdx.x == 0) p.parts[(batch * p.bands + band) * p.runs + run] = sum;
  for (int i = threadIdx.x; i < kNormRun && n0 + i < p.N; i += 256)
    p.col_parts[(batch * p.bands + band) * p.N + n0 + i] =
        max(max(tops[0][i], tops[1][i]), max(tops[2][i], tops[3][i]));
}

// The largest of `count` numbers `step` apart, of which kTogether are loaded together.
template <int kTogether>
__device__ __forceinline__ unsigned top_of(const unsigned *part, int count, long step) {
  unsigned top = 0;
  for (int k = 0; k < count; k += kTogether) {
    unsigned v[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) v[j] = part[min(k + j, count - 1) * step];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) top = max(top, v[j]);
  }
  return top;
}

// What X is multiplied by, from the parts of its sum of squares.
__device__ __forceinline__ double scale_of(const OrthoSizesArgs &p, long batch) {
  const int all = p.bands * p.runs;
  double sum = 0;
  for (int k = threadIdx.x; k < all; k += 256) sum += p.parts[batch * all + k];
  const double norm = sqrt(group_sum(sum)) + (double)p.eps;
  return norm > 0 ? 1.0 / norm : norm;  // NaN stays
}

__device__ __forceinline__ signed char scaled_exponent(unsigned top, double scale, int length) {
  const float size = (float)(scale * (double)__uint_as_float(top));
  return norm_exponent(__float_as_uint(size) & 0x7fffffffu, length);
}

// For very long rows or columns, whose sizes are in so many parts that each block of the
// next launch would not add them up for itself: a thread has a row or a column, or
// the 2^shift that share an exponent.
__global__ void __launch_bounds__(256) ortho_scales_kernel(OrthoSizesArgs p) {
  const long batch = blockIdx.y;
  const int row_count = ((p.M - 1) >> p.row_shift) + 1, col_count = ((p.N - 1) >> p.col_shift) + 1;
  const int row_groups = (row_count + 255) / 256;
  const bool of_rows = (int)blockIdx.x < row_groups;
  const int i = ((int)blockIdx.x - (of_rows ? 0 : row_groups)) * 256 + (int)threadIdx.x;
  const int count = of_rows ? row_count : col_count, shift = of_rows ? p.row_shift : p.col_shift;
  const int n = of_rows ? p.M : p.N, parts = of_rows ? p.runs : p.bands;
  const unsigned *const from = (of_rows ? p.row_parts : p.col_parts) + batch * parts * n;
  unsigned top = 0;
  for (int k = 0; k < 1 << shift; ++k)
    top = max(top, top_of<32>(from + min((min(i, count - 1) << shift) + k, n - 1), parts, n));
  const double scale = p.scale ? scale_of(p, batch) : 1.0;
  if (p.scale && blockIdx.x == 0 && threadIdx.x == 0) p.scale[batch] = scale;
  if (i < count)
    (of_rows ? p.rows : p.cols)[batch * count + i] =
        scaled_exponent(top, scale, of_rows ? p.row_length : p.col_length);
}

__global__ void __launch_bounds__(256) ortho_clear_kernel(unsigned *at, long n) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) at[i] = 0;
}

// The largest magnitudes of the rows and columns of a held matrix, into zeros: 4 lanes have
// 32 columns of a row, a work-group kLookRows rows, 64 at a time.
constexpr int kLookRows = 512;
__global__ void __launch_bounds__(256) ortho_look_kernel(SplitMatrix z, RowScale by, unsigned *rows,
                                                         unsigned *cols) {
  const int lane = threadIdx.x % kWave, part = threadIdx.x % 4;
  const int c0 = blockIdx.y * 32, first = (int)blockIdx.x * kLookRows;
  const long batch = blockIdx.z;
  float top[8];  // of the lane's columns
#pragma unroll
  for (int e = 0; e < 8; ++e) top[e] = 0.f;
  for (int r0 = first; r0 < min(first + kLookRows, z.rows); r0 += 64) {
    const int r = r0 + (int)threadIdx.x / 4;
    float most = 0.f;
    if (r < z.rows) {
      const f16x8 high =
          *reinterpret_cast<const f16x8 *>(z.place(blockIdx.z, r, c0) + part * 16);
      const float scale = power_of_two(by.exponent(by.norm[by.index(batch, r)]) - kHeldTop);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float size = fabsf((float)high[e]) * scale;
        top[e] = fmaxf(top[e], size);
        most = fmaxf(most, size);
      }
    }
    most = fmaxf(most, __shfl_xor(most, 1));
    most = fmaxf(most, __shfl_xor(most, 2));
    if (r < z.rows && part == 0) atomicMax(rows + batch * z.rows + r, __float_as_uint(most));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int d = 32; d > 2; d /= 2) top[e] = fmaxf(top[e], __shfl_xor(top[e], d));
    const int c = c0 + part * 8 + e;
    if (lane < 4 && c < z.cols) atomicMax(cols + batch * z.cols + c, __float_as_uint(top[e]));
  }
}

// A block of 32 x 32 per wave, in the layout of the matrix instructions' results: lane
// l has column l % 32 of rows 8 q + 4 (l / 32) .. + 3.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_split_kernel(OrthoSplitArgs p, FastDiv by_across) {
  const OrthoSizesArgs &x = p.x;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int block = blockIdx.x * 4 + wave, row = by_across(block);
  const int bm = row * 32, bn = (block - row * ((x.N + 31) / 32)) * 32;
  const int r32 = lane % 32, half = lane / 32;
  const long batch = blockIdx.y;
  // Every lane loads, from the nearest element there is, so that the loads go out
  // together; what lies past the matrix is then dropped.
  float v[16];
  const int n = min(bn + r32, x.N - 1);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int m = min(bm + acc32_row(lane, e), x.M - 1);
    v[e] = load1<BF16>(x.X, batch * x.strideX + m * x.ldx + n);
  }
  // A lane has the exponent of a row, or of a column.
  const bool of_rows = half == 0;
  const RowScale by = either(of_rows, p.row_scale, p.col_scale);
  const int i = of_rows ? min(bm + r32, x.M - 1) : n;
  double scale;
  int norm;
  if (x.summed) {
    scale = x.scale[batch];
    norm = by.norm[by.index(batch, i)];
  } else {
    const int parts = of_rows ? x.runs : x.bands, length = of_rows ? x.M : x.N;
    const unsigned top = top_of<8>(
        (of_rows ? x.row_parts : x.col_parts) + batch * parts * length + i, parts, length);
    scale = scale_of(x, batch);
    const signed char e = scaled_exponent(top, scale, of_rows ? x.row_length : x.col_length);
    if (of_rows ? bn == 0 && bm + r32 < x.M : bm == 0 && bn + r32 < x.N)
      (of_rows ? x.rows : x.cols)[batch * length + i] = e;
    norm = e;
  }
  if (bm >= x.M) return;  // whole waves: no barrier follows
  __shared__ __attribute__((aligned(16))) float scales[4][2][32];
  scales[wave][half][r32] = power_of_two(kHeldTop - by.exponent(norm));
  wave_fence();
  float row_scale[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f32x4 r = *reinterpret_cast<const f32x4 *>(&scales[wave][0][8 * q + 4 * half]);
#pragma unroll
    for (int e = 0; e < 4; ++e) row_scale[4 * q + e] = r[e];
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const bool in = bm + acc32_row(lane, e) < x.M && bn + r32 < x.N;
    v[e] = in ? (float)(scale * (double)v[e]) : 0.f;
  }
  __shared__ __attribute__((aligned(16))) char images[4][2][4096];
  const BlockImage rows{images[wave][0]}, cols{images[wave][1]};
  split_block(v, row_scale, r32, half, rows);
  split_transposed(v, scales[wave][1][r32], r32, half, cols);
  wave_fence();
  store_block(p.rows, blockIdx.y, bm, bn, x.M, lane, rows);
  store_block(p.cols, blockIdx.y, bn, bm, x.N, lane, cols);
}

// Position `id` of the tiles on and below a diagonal, row by row: row t has t + 1.
__device__ __forceinline__ void triangle_tile(int id, int &tm, int &tn) {
  int t = (int)((sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
  while (t * (t + 1) / 2 > id) --t;
  while ((t + 1) * (t + 2) / 2 <= id) ++t;
  tm = t;
  tn = id - t * (t + 1) / 2;
}

// The epilogue moves whole blocks of 32 x 32 between memory and LDS, 16 bytes a lane
// and 1 KiB of consecutive bytes an instruction.  Straight from the registers' layout,
// with 2 and 8 bytes a lane over rows 128 bytes apart, E and the two results took
// 45 of 105 us of a 2048 x 4096 x 2048 product.
template <int BM, int BN, int WM, int WN, int NST, bool SYMMETRIC>
__global__ void __launch_bounds__(WM *WN *kWave, 2)
ortho_product_kernel(OrthoProductArgs p, TileMap map, FastDiv by_triangle, int triangle,
                     bool y_bf16) {
  using Tile = SliceTile<SplitFormat, BM, BN, WM, WN, NST>;
  constexpr int FM = Tile::FM, FN = Tile::FN;
  static_assert(Tile::STAGE_BYTES >= WM * WN * 4096 && NST >= 3, "a block per wave and image");
  const int lane = threadIdx.x % kWave, r32 = lane % 32, half = lane / 32;
  const int id = xcd_contiguous_id(blockIdx.x, gridDim.x);
  int batch, tm, tn;
  if constexpr (SYMMETRIC) {
    batch = by_triangle(id);
    triangle_tile(id - batch * triangle, tm, tn);
  } else {
    map.tile(id, batch, tm, tn);
  }
  const int m0 = tm * BM, n0 = tn * BN;
  const int M = p.a.rows, N = p.b.rows;
  const int rows_a = min(BM, M - m0), rows_b = min(BN, N - n0);
  const int mw = m0 + Tile::row0(), nw = n0 + Tile::col0();

  // Blocks of E^T go out before the sums' operands; rows past N are zeros, and a row's
  // columns up to the next 32 are there.
  slice_i32x4 e_t[FM][FN][4];
  const bool whole = mw + 32 * FM <= M && nw + 32 * FN <= N;
  auto load_e = [&](const SplitMatrix &x, int r0, int c, int k) {
    const int r = r0 + 8 * k + lane / 8;
    const auto *at = reinterpret_cast<const slice_i32x4 *>(x.place(batch, r, c) + lane % 8 * 16);
    if (whole) return *at;
    return r < x.rows && c < x.cols ? *at : slice_i32x4{0, 0, 0, 0};
  };
  if (p.e.at) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) e_t[i][j][k] = load_e(p.e_t, nw + j * 32, mw + i * 32, k);
  }

  auto rows = [&](const SplitMatrix &x, int first, int n) {
    return SliceRows{x.place(batch, first, 0), kSliceRow, (long)x.rows * kSliceRow, n};
  };
  // A thread has a row of A or of B: the norms that its scales go by are loaded here, and
  // waited for while the first slices come.  The threads there are more do the same, for
  // nothing: behind a test the compiler would load them there, after the slices.
  static_assert(BM + BN <= Tile::kThreads, "a thread for each row");
  const bool of_a = threadIdx.x < BM;
  const int own = of_a ? min(m0 + (int)threadIdx.x, M - 1) : min(n0 + (int)threadIdx.x - BM, N - 1);
  const RowScale from = either(of_a, p.a_scale, p.b_scale), to = either(of_a, p.d_scale, p.d_t_scale),
                 of_e = either(of_a, p.e_scale, p.b_scale);
  auto norm_of = [&](const RowScale &x) -> int {
    return x.norm[x.index(batch, own)];
  };
  const int norm_in = norm_of(from), norm_out = norm_of(to), norm_e = norm_of(of_e);

  // What a row's and a column's sums are multiplied by, and the powers of two under which
  // the results, and E's rows, are held; and of every 32 rows the least exponent of E's,
  // negative, of every 32 columns the largest.
  __shared__ __attribute__((aligned(16))) float in_scales[Tile::kThreads],
      out_scales[Tile::kThreads], e_scales[Tile::kThreads];
  __shared__ int ranges[Tile::kThreads / 32];
  auto keep_scales = [&] {
    const int e = of_e.exponent(norm_e);
    in_scales[threadIdx.x] = power_of_two(from.exponent(norm_in) - kHeldTop) * (of_a ? p.f1 : 1.f);
    out_scales[threadIdx.x] = power_of_two(kHeldTop - to.exponent(norm_out));
    e_scales[threadIdx.x] = power_of_two(e - kHeldTop);
    const int top = half_wave_max(of_a ? -e : e);
    if (r32 == 31) ranges[threadIdx.x / 32] = top;
  };
  f32x16 acc[FM][FN];
  char *lds[NST];
  Tile::run(rows(p.a, m0, rows_a), rows(p.b, n0, rows_b), (p.a.cols + 31) / 32, acc, lds,
            keep_scales);
  __syncthreads();  // no loads into the stages are left, of any wave
  const int wave = Tile::wave_id();
  const BlockImage e_image{lds[0] + wave * 4096}, t_image{lds[1] + wave * 4096},
      d_image{lds[2] + wave * 4096};

  // Register e of lane l holds row acc32_row(l, e), column l % 32 of a block: four
  // rows 8 q + 4 (l / 32) .. + 3, which are neighbours in a transposed matrix.
  const SplitMatrix &t = SYMMETRIC ? p.d : p.d_t;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int mb = mw + i * 32, nb = nw + j * 32;  // the block's origin
      if (mb >= M || nb >= N) continue;
      // Blocks above the diagonal come from below it, in whatever tile they lie: an
      // element's terms are added in the same order with every tile.
      if (SYMMETRIC && mb < nb) continue;
      const bool mirror = t.at && (!SYMMETRIC || mb > nb);
      float v[16], scale_out[16];
      const int of_b = BM + Tile::col0() + j * 32 + r32;
      const float scale_b = in_scales[of_b];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = Tile::row0() + i * 32 + 8 * q + 4 * half;
        const f32x4 in = *reinterpret_cast<const f32x4 *>(in_scales + at);
        const f32x4 out = *reinterpret_cast<const f32x4 *>(out_scales + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[4 * q + e] = acc[i][j][4 * q + e] * scale_b * in[e];
          scale_out[4 * q + e] = out[e];
        }
      }
      if (p.e.at) {
        // By columns, where none of them has a range 2^8 times that of a row: what is held to
        // 2^-40 of its column is then held to 2^-32 of its row too.  Read by rows as well (all
        // blocks, every other row 1e-6 of the next): 2048 x 4096 1027 us for 997.
        const bool by_rows = __builtin_amdgcn_readfirstlane(
            ranges[Tile::row0() / 32 + i] + ranges[(BM + Tile::col0()) / 32 + j] > 8);
#pragma unroll
        for (int k = 0; k < 4; ++k) *e_image.linear(lane, k) = e_t[i][j][k];
        if (by_rows) {
#pragma unroll 1  // rarely: no registers are spent on it
          for (int k = 0; k < 4; ++k) *t_image.linear(lane, k) = load_e(p.e, mb, nb, k);
        }
        wave_fence();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f16x4 high = *reinterpret_cast<const f16x4 *>(e_image.chunk(r32, q) + 8 * half);
          const f16x4 low = *reinterpret_cast<const f16x4 *>(e_image.chunk(r32, 4 + q) + 8 * half);
          f32x4 value;
#pragma unroll
          for (int e = 0; e < 4; ++e) value[e] = ((float)high[e] + (float)low[e]) * scale_b;
          if (by_rows) {
            const int m = 8 * q + 4 * half;
            const f32x4 scale_e =
                *reinterpret_cast<const f32x4 *>(e_scales + Tile::row0() + i * 32 + m);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const auto piece = [&](int c) {
                return (float)reinterpret_cast<_Float16 *>(t_image.chunk(m + e, c + r32 / 8))[r32 % 8];
              };
              if (scale_e[e] < scale_b) value[e] = (piece(0) + piece(4)) * scale_e[e];
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] = fmaf(p.f2, value[e], v[4 * q + e]);
        }
      }
      wave_fence();
      if (!SYMMETRIC && p.Y) {
        // Floats, as the user's rows run: 32 of them are 128 bytes too.
        const bool turned = p.y_transposed;
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= p.alpha;
        floats_block(v, turned, r32, half, d_image);
        wave_fence();
        const int r0 = turned ? nb : mb, c0 = (turned ? mb : nb) + lane % 8 * 4;
        const int rows = turned ? N : M, left = (turned ? M : N) - c0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = r0 + 8 * k + lane / 8;
          const f32x4 w = __builtin_bit_cast(f32x4, *d_image.linear(lane, k));
          if (r >= rows) continue;
          const long at = batch * p.strideY + r * p.ldy + c0;
          if (y_bf16) {
            __bf16 *y = static_cast<__bf16 *>(p.Y) + at;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < left) y[e] = (__bf16)w[e];
          } else {
            float *y = static_cast<float *>(p.Y) + at;
            if (left >= 4) {
              *reinterpret_cast<f32x4_any *>(y) = w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (e < left) y[e] = w[e];
            }
          }
        }
        wave_fence();
        continue;
      }
      split_block(v, scale_out, r32, half, d_image);
      if (mirror) split_transposed(v, out_scales[of_b], r32, half, t_image);
      wave_fence();
      // Rows of a result are written up to the end of their last 32 columns: past
      // its own columns the sums are 0.
      store_block(p.d, batch, mb, nb, M, lane, d_image);
      if (mirror) store_block(t, batch, nb, mb, N, lane, t_image);
      wave_fence();
    }
  for (unsigned at = blockIdx.x * Tile::kThreads + threadIdx.x; at < p.moves;
       at += gridDim.x * Tile::kThreads)
    reinterpret_cast<slice_i32x4 *>(p.move_to)[at] =
        reinterpret_cast<const slice_i32x4 *>(p.move_from)[at];
}

template <int BM, int BN, int WM, int WN, int NST>
hipError_t launch(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                  hipStream_t s) {
  const int tiles_m = (p.a.rows + BM - 1) / BM, tiles_n = (p.b.rows + BN - 1) / BN;
  const TileMap map = make_tile_map(tiles_m, tiles_n, 8);
  const dim3 block(WM * WN * kWave);
  if constexpr (BM == BN) {
    if (symmetric) {
      const int triangle = tiles_m * (tiles_m + 1) / 2;
      hipLaunchKernelGGL((ortho_product_kernel<BM, BN, WM, WN, NST, true>),
                         dim3((unsigned)(triangle * batch)), block, 0, s, p, map,
                         make_fast_div(triangle), triangle, y_bf16);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((ortho_product_kernel<BM, BN, WM, WN, NST, false>),
                     dim3((unsigned)((long)tiles_m * tiles_n * batch)), block, 0, s, p, map,
                     make_fast_div(1), 1, y_bf16);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ortho_norm(const OrthoNormArgs &p, bool bf16, int batch, hipStream_t s) {
  const dim3 grid((unsigned)p.n_parts, (unsigned)batch), block(256);
  if (bf16)
    hipLaunchKernelGGL(ortho_norm_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(ortho_norm_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

namespace {

hipError_t launch_scales(const OrthoSizesArgs &p, int batch, hipStream_t s) {
  const int rows = ((p.M - 1) >> p.row_shift) + 1, cols = ((p.N - 1) >> p.col_shift) + 1;
  const dim3 grid((unsigned)((rows + 255) / 256 + (cols + 255) / 256), (unsigned)batch);
  hipLaunchKernelGGL(ortho_scales_kernel, grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ortho_sizes(const OrthoSizesArgs &p, bool bf16, int batch, hipStream_t s) {
  const dim3 block(256), grid((unsigned)((long)p.bands * p.runs), (unsigned)batch);
  if (bf16)
    hipLaunchKernelGGL(ortho_sizes_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(ortho_sizes_kernel<false>, grid, block, 0, s, p);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess || !p.summed ? err : launch_scales(p, batch, s);
}

hipError_t launch_ortho_look(const OrthoSizesArgs &p, const SplitMatrix &z, const RowScale &z_scale,
                             int batch, hipStream_t s) {
  const long tops = (long)batch * (p.M + p.N);
  hipLaunchKernelGGL(ortho_clear_kernel, dim3((unsigned)((tops + 255) / 256)), dim3(256), 0, s,
                     p.row_parts, tops);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)((z.rows + kLookRows - 1) / kLookRows), (unsigned)((z.cols + 31) / 32),
                  (unsigned)batch);
  hipLaunchKernelGGL(ortho_look_kernel, grid, dim3(256), 0, s, z, z_scale, p.row_parts, p.col_parts);
  err = hipGetLastError();
  return err != hipSuccess ? err : launch_scales(p, batch, s);
}

hipError_t launch_ortho_split(const OrthoSplitArgs &p, bool bf16, int batch, hipStream_t s) {
  const long blocks = ((p.x.M + 31L) / 32) * ((p.x.N + 31L) / 32);
  const dim3 grid((unsigned)((blocks + 3) / 4), (unsigned)batch), block(256);
  const FastDiv by_across = make_fast_div((p.x.N + 31) / 32);
  if (bf16)
    hipLaunchKernelGGL(ortho_split_kernel<true>, grid, block, 0, s, p, by_across);
  else
    hipLaunchKernelGGL(ortho_split_kernel<false>, grid, block, 0, s, p, by_across);
  return hipGetLastError();
}

hipError_t launch_ortho_product(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                                int cus, hipStream_t s) {
  const OrthoTile tile = ortho_tile(p.a.rows, p.b.rows, p.a.cols, symmetric, batch, cus);
  if (tile == OrthoTile::k64) return launch<64, 64, 2, 2, 4>(p, symmetric, y_bf16, batch, s);
  return tile == OrthoTile::k128 ? launch<128, 128, 2, 4, 3>(p, symmetric, y_bf16, batch, s)
                                 : launch<128, 256, 2, 4, 3>(p, false, y_bf16, batch, s);
}

}  // namespace sgemm
