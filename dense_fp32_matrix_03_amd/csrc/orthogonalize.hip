// orthogonalize.hip -- the products of Newton-Schulz steps
// (include/sgemm_orthogonalize.h) on the half-precision matrix cores.
//
// A value v is held as high + low, two half-precision numbers, high = v rounded and
// low = v - high rounded: off by 2^-22 of v at most.  A product a b is then
// al bh + ah bl + ah bh, three instructions instead of one (al bl, below 2^-22 of
// it, is left out).  All matrices are scaled by powers of two so that the largest
// element that their singular values allow stays below 2^15.
//
// With m <= n a step is S = Z Z^T, P = b S + c S S and a Z + P Z.  All three are
// products of rows by rows once Z is held transposed too: the epilogue writes a
// result as it is and transposed.  S and P are symmetric: tiles on and below the
// diagonal are computed, and written to both sides.
//
// Three times the operations of the formula at half precision's rate (1.33 PFLOP/s in a
// large library product) are the floor.  Five steps, microseconds and the floor:
//   1 x 2048 x 4096      945 - 965   676    the power limit: a Z + P Z 92 (1.12 PFLOP/s), S
//                                           48 - 60 and P 37 (136 tiles on 256 compute units)
//   1 x 1500 x 1001      200          62    S and P 11 each, a Z + P Z 17.5: 1.5 rounds of
//                                           tiles, fixed costs of 4 to 5 us a launch
//   16 x 256 x 512       115          21    17 launches of 4 to 11 us, of which 4 to 5 are
//                                           fixed: first loads from memory, and the stores
// The norm and the split are bound by memory: 2048 x 4096 9.1 us (3.7 TB/s) and 16.5 (6.1).
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

// The pieces of a block of sums (as the matrix instructions leave them) to images of
// the block and, with `both`, of its transpose.
__device__ __forceinline__ void split_block(const float v[16], int r32, int half,
                                            const BlockImage &d, const BlockImage &t, bool both) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f16x4 high, low;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      _Float16 h, l;
      split(v[4 * q + e], h, l);
      high[e] = h;
      low[e] = l;
      const int m = 8 * q + 4 * half + e;
      reinterpret_cast<_Float16 *>(d.chunk(m, r32 / 8))[r32 % 8] = h;
      reinterpret_cast<_Float16 *>(d.chunk(m, 4 + r32 / 8))[r32 % 8] = l;
    }
    if (both) {
      *reinterpret_cast<f16x4 *>(t.chunk(r32, q) + 8 * half) = high;
      *reinterpret_cast<f16x4 *>(t.chunk(r32, 4 + q) + 8 * half) = low;
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

// A block of 32 x 32 per wave, in the layout of the matrix instructions' results: lane
// l has column l % 32 of rows 8 q + 4 (l / 32) .. + 3.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_split_kernel(OrthoSplitArgs p, FastDiv by_across) {
  const OrthoNormArgs &x = p.x;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const double part = (int)threadIdx.x < x.n_parts
                          ? x.parts[(long)blockIdx.y * x.n_parts + threadIdx.x] : 0.0;
  const int block = blockIdx.x * 4 + wave, row = by_across(block);
  const int bm = row * 32, bn = (block - row * ((x.N + 31) / 32)) * 32;
  const int r32 = lane % 32, half = lane / 32;
  // Every lane loads, from the nearest element there is, so that the loads go out
  // together; what lies past the matrix is then dropped.
  float v[16];
  const int n = bn + r32;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int m = min(bm + acc32_row(lane, e), x.M - 1);
    v[e] = load1<BF16>(x.X, (long)blockIdx.y * x.strideX + m * x.ldx + min(n, x.N - 1));
  }
  const double norm = sqrt(group_sum(part)) + (double)p.eps;
  const double scale = norm > 0 ? ldexp(1.0, p.shift) / norm : norm;  // NaN stays
  if (bm >= x.M) return;  // whole waves: no barrier follows
#pragma unroll
  for (int e = 0; e < 16; ++e)
    v[e] = bm + acc32_row(lane, e) < x.M && n < x.N ? (float)(scale * (double)v[e]) : 0.f;
  __shared__ __attribute__((aligned(16))) char images[4][2][4096];
  const BlockImage rows{images[wave][0]}, cols{images[wave][1]};
  split_block(v, r32, half, rows, cols, true);
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
  auto load_e = [&](bool whole) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = nw + j * 32 + 8 * k + lane / 8, m = mw + i * 32;
          const auto *at =
              reinterpret_cast<const slice_i32x4 *>(p.e_t.place(batch, n, m) + lane % 8 * 16);
          if (whole)
            e_t[i][j][k] = *at;
          else
            e_t[i][j][k] = n < N && m < M ? *at : slice_i32x4{0, 0, 0, 0};
        }
  };
  if (p.e_t.at) load_e(mw + 32 * FM <= M && nw + 32 * FN <= N);

  auto rows = [&](const SplitMatrix &x, int first, int n) {
    return SliceRows{x.place(batch, first, 0), kSliceRow, (long)x.rows * kSliceRow, n};
  };
  f32x16 acc[FM][FN];
  char *lds[NST];
  Tile::run(rows(p.a, m0, rows_a), rows(p.b, n0, rows_b), (p.a.cols + 31) / 32, acc, lds);
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
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = p.f1 * acc[i][j][e];
      if (p.e_t.at) {
#pragma unroll
        for (int k = 0; k < 4; ++k) *e_image.linear(lane, k) = e_t[i][j][k];
        wave_fence();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f16x4 high = *reinterpret_cast<const f16x4 *>(e_image.chunk(r32, q) + 8 * half);
          const f16x4 low = *reinterpret_cast<const f16x4 *>(e_image.chunk(r32, 4 + q) + 8 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[4 * q + e] = fmaf(p.f2, (float)high[e] + (float)low[e], v[4 * q + e]);
        }
        wave_fence();
      }
      if (p.Y) {
        // Floats, as the user's rows run: 32 of them are 128 bytes too.
        const bool turned = p.y_transposed;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = 8 * q + 4 * half;
          if (turned) {
            *reinterpret_cast<f32x4 *>(d_image.chunk(r32, m / 4)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<float *>(d_image.chunk(m + e, r32 / 4))[r32 % 4] = v[4 * q + e];
          }
        }
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
      split_block(v, r32, half, d_image, t_image, mirror);
      wave_fence();
      // Rows of a result are written up to the end of their last 32 columns: past
      // its own columns the sums are 0.
      store_block(p.d, batch, mb, nb, M, lane, d_image);
      if (mirror) store_block(t, batch, nb, mb, N, lane, t_image);
      wave_fence();
    }
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

// The tile by times in microseconds, n the tiles for each of the chip's compute units,
// nk slices.  Measured on 256 compute units (S = Z Z^T, or a Z + P Z; m x n of Z, tiles
// of 64 x 64 / 128 x 128 / 128 x 256):
//   S    1024 x 1024      10.0 / 18.8       2048 x 2048      45 / 41
//        2600 x 2600      91 / 58           2048 x 4096      80 / 58
//        16 of 512 x 512  17.5 / 16.1       1500 x 1500      22 / 26
//   a Z + P Z
//        1024 x 1024      13.3 / 22 / 34    2048 x 2048      64 / 54 / 69
//        2600 x 2600      132 / 116 / 107   2048 x 4096      122 / 103 / 92
//        16 of 512 x 512  28 / 24 / 29      1500 x 1500      36 / 32 / 47
// A tile of 64 x 64 is bound by what the caches deliver, 85 bytes a nanosecond and
// compute unit; larger ones by the matrix cores, at the power limit once the chip is
// full (1.1 PFLOP/s of half precision, where a large library product has 1.3).
hipError_t launch_ortho_product(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                                int cus, hipStream_t s) {
  const double nk = (p.a.cols + 31) / 32;
  auto tiles = [&](int bm, int bn) {
    const double tm = (p.a.rows + bm - 1) / bm, tn = (p.b.rows + bn - 1) / bn;
    return batch * (symmetric ? tm * (tm + 1) / 2 : tm * tn) / cus;
  };
  const double n64 = tiles(64, 64), n128 = tiles(128, 128);
  const double c64 = ceil(n64) * (0.2 * nk + 2);
  if (symmetric) {
    const double c128 = ceil(n128) * (0.38 * nk + 6 + 12 * fmin(n128, 1));
    return c64 <= c128 ? launch<64, 64, 2, 2, 4>(p, true, y_bf16, batch, s)
                       : launch<128, 128, 2, 4, 3>(p, true, y_bf16, batch, s);
  }
  const double c128 =
      fmax(1, (ceil(n128) + n128) / 2) * ((0.38 + 0.22 * fmin(n128, 1)) * nk + 11);
  const double n256 = tiles(128, 256);
  const double c256 = ceil(n256) * (0.85 * nk + 12 + 50 * fmin(fmax(n256 - 0.6, 0), 0.4));
  if (c64 <= c128 && c64 <= c256) return launch<64, 64, 2, 2, 4>(p, false, y_bf16, batch, s);
  return c128 <= c256 ? launch<128, 128, 2, 4, 3>(p, false, y_bf16, batch, s)
                      : launch<128, 256, 2, 4, 3>(p, false, y_bf16, batch, s);
}

}  // namespace sgemm
