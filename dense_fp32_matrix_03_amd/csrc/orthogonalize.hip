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
#include "mxfp4.hpp"
#include "orthogonalize.hpp"
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
  static constexpr int kSteps = 2, kReads = 2, kMfma = 3;
  template <int S, class At>
  __device__ __forceinline__ static Frag load(int half, At at) {
    return {__builtin_bit_cast(f16x8, *at(2 * S + half)),
            __builtin_bit_cast(f16x8, *at(4 + 2 * S + half))};
  }
  __device__ __forceinline__ static void mma(const Frag &a, const Frag &b, Acc &c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.low, b.high, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.high, b.low, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.high, b.high, c, 0, 0, 0);
  }
};

__device__ __forceinline__ void split(float v, _Float16 &high, _Float16 &low) {
  high = (_Float16)v;
  low = (_Float16)(v - (float)high);
}

// Where column c of a row lies: its high piece, the low one 64 bytes after it.
__device__ __forceinline__ long split_at(int c) { return (long)(c / 32) * 128 + c % 32 * 2; }

template <bool BF16>
__device__ __forceinline__ float load1(const void *x, long at) {
  if constexpr (BF16)
    return __uint_as_float((unsigned)static_cast<const unsigned short *>(x)[at] << 16);
  else
    return static_cast<const float *>(x)[at];
}

__device__ __forceinline__ double group_sum(double v) {  // of 256 threads
  __shared__ double part[4];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  return part[0] + part[1] + part[2] + part[3];
}

// Part blockIdx.x of matrix blockIdx.y: every n_parts-th run of 2048 elements.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_norm_kernel(OrthoNormArgs p) {
  const long base = (long)blockIdx.y * p.strideX;
  const int runs = (p.N + 2047) / 2048;
  double sum = 0;
  for (long u = blockIdx.x; u < (long)p.M * runs; u += p.n_parts) {
    const long row = u / runs;
    const int n = (int)(u - row * runs) * 2048 + threadIdx.x * 8;
    float v[8];
    load8<BF16>(static_cast<const char *>(p.X) + (base + row * p.ldx + n) * (BF16 ? 2 : 4),
                p.N - n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += (double)v[e] * (double)v[e];
  }
  sum = group_sum(sum);
  if (threadIdx.x == 0) p.parts[(long)blockIdx.y * p.n_parts + blockIdx.x] = sum;
}

// A block of 32 x 32 per wave: lane l has column l % 32 of rows l / 32, + 2, ...
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_split_kernel(OrthoSplitArgs p) {
  const OrthoNormArgs &x = p.x;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const double part = (int)threadIdx.x < x.n_parts
                          ? x.parts[(long)blockIdx.y * x.n_parts + threadIdx.x] : 0.0;
  const double norm = sqrt(group_sum(part)) + (double)p.eps;
  const double scale = norm > 0 ? ldexp(1.0, p.shift) / norm : norm;  // NaN stays
  __shared__ float tile[4][32][33];
  const int across = (x.N + 31) / 32, down = (x.M + 31) / 32;
  const long block = (long)blockIdx.x * 4 + wave;
  const int bm = (int)(block / across), bn = (int)(block - (long)bm * across);
  if (bm >= down) return;  // whole waves: no barrier follows
  const int c = lane % 32, r0 = lane / 32;
  char *const rows = p.rows.at + blockIdx.y * p.rows.stride;
  char *const cols = p.cols.at + blockIdx.y * p.cols.stride;
  auto store = [&](char *to, float v) {
    _Float16 high, low;
    split(v, high, low);
    *reinterpret_cast<_Float16 *>(to) = high;
    *reinterpret_cast<_Float16 *>(to + 64) = low;
  };
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = r0 + 2 * i, m = bm * 32 + r, n = bn * 32 + c;
    float v = 0.f;
    if (m < x.M && n < x.N)
      v = (float)(scale * (double)load1<BF16>(x.X, (long)blockIdx.y * x.strideX + m * x.ldx + n));
    tile[wave][r][c] = v;
    if (m < x.M) store(rows + (long)m * p.rows.pitch + bn * 128 + c * 2, v);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = r0 + 2 * i, n = bn * 32 + r;
    if (n < x.N) store(cols + (long)n * p.cols.pitch + bm * 128 + c * 2, tile[wave][c][r]);
  }
}

// Position `id` of the tiles on and below a diagonal, row by row: row t has t + 1.
__device__ __forceinline__ void triangle_tile(int id, int &tm, int &tn) {
  int t = (int)((sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
  while (t * (t + 1) / 2 > id) --t;
  while ((t + 1) * (t + 2) / 2 <= id) ++t;
  tm = t;
  tn = id - t * (t + 1) / 2;
}

template <int BM, int BN, int WM, int WN, int KS, bool SYMMETRIC>
__global__ void __launch_bounds__(WM *WN *KS *kWave, 2)
ortho_product_kernel(OrthoProductArgs p, TileMap map, FastDiv by_triangle, int triangle,
                     bool y_bf16) {
  using Tile = SliceTile<SplitFormat, BM, BN, WM, WN, KS>;
  constexpr int FM = Tile::FM, FN = Tile::FN;
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
  f32x16 acc[FM][FN];
  if (!Tile::run(p.a.at + batch * p.a.stride + (long)m0 * p.a.pitch, p.a.pitch, rows_a,
                 p.b.at + batch * p.b.stride + (long)n0 * p.b.pitch, p.b.pitch, rows_b,
                 p.a.pitch / kSliceRow, acc))
    return;

  // Register e of lane l holds row acc32_row(l, e), column l % 32 of a block: four
  // rows 8 q + 4 (l / 32) .. + 3, which are neighbours in a transposed matrix.
  const int mw = m0 + Tile::row0(), nw = n0 + Tile::col0() + r32;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = nw + j * 32;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = mw + i * 32 + 8 * q + 4 * half;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p.f1 * acc[i][j][4 * q + e];
        if (p.e_t.at && n < N && m < M) {  // columns up to the next 32 are there
          const char *at = p.e_t.at + batch * p.e_t.stride + (long)n * p.e_t.pitch + split_at(m);
          const f16x4 high = *reinterpret_cast<const f16x4 *>(at);
          const f16x4 low = *reinterpret_cast<const f16x4 *>(at + 64);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = fmaf(p.f2, (float)high[e] + (float)low[e], v[e]);
        }
        if (p.Y) {
          if (n >= N) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (m + e >= M) continue;
            const long at = batch * p.strideY + (p.y_transposed ? n * p.ldy + m + e
                                                               : (m + e) * p.ldy + n);
            if (y_bf16)
              static_cast<__bf16 *>(p.Y)[at] = (__bf16)v[e];
            else
              static_cast<float *>(p.Y)[at] = v[e];
          }
          continue;
        }
        f16x4 high, low;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          _Float16 h, l;
          split(v[e], h, l);
          high[e] = h;
          low[e] = l;
        }
        // Rows of a result are written up to the end of their last 32 columns: past
        // its own columns the sums are 0.
        if (p.d.at && n < p.d.pitch / 4) {
          char *at = p.d.at + batch * p.d.stride + (long)m * p.d.pitch + split_at(n);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (m + e >= M) continue;
            *reinterpret_cast<_Float16 *>(at + (long)e * p.d.pitch) = high[e];
            *reinterpret_cast<_Float16 *>(at + (long)e * p.d.pitch + 64) = low[e];
          }
        }
        const SplitMatrix &t = SYMMETRIC ? p.d : p.d_t;
        if (t.at && n < N && m < t.pitch / 4 && (!SYMMETRIC || tm != tn)) {
          char *at = t.at + batch * t.stride + (long)n * t.pitch + split_at(m);
          *reinterpret_cast<f16x4 *>(at) = high;
          *reinterpret_cast<f16x4 *>(at + 64) = low;
        }
      }
    }
}

template <int BM, int BN, int WM, int WN, int KS>
hipError_t launch(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                  hipStream_t s) {
  const int tiles_m = (p.a.rows + BM - 1) / BM, tiles_n = (p.b.rows + BN - 1) / BN;
  const int triangle = symmetric ? tiles_m * (tiles_m + 1) / 2 : 1;
  const TileMap map = make_tile_map(tiles_m, tiles_n, 8);
  const dim3 block(WM * WN * KS * kWave);
  if (symmetric)
    hipLaunchKernelGGL((ortho_product_kernel<BM, BN, WM, WN, KS, true>),
                       dim3((unsigned)(triangle * batch)), block, 0, s, p, map,
                       make_fast_div(triangle), triangle, y_bf16);
  else
    hipLaunchKernelGGL((ortho_product_kernel<BM, BN, WM, WN, KS, false>),
                       dim3((unsigned)((long)tiles_m * tiles_n * batch)), block, 0, s, p, map,
                       make_fast_div(1), triangle, y_bf16);
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
  if (bf16)
    hipLaunchKernelGGL(ortho_split_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(ortho_split_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_ortho_product(const OrthoProductArgs &p, bool symmetric, bool y_bf16, int batch,
                                int, hipStream_t s) {
  return launch<64, 64, 2, 2, 1>(p, symmetric, y_bf16, batch, s);
}

}  // namespace sgemm
