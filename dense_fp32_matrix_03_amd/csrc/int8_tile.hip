// int8_tile.hip -- products of matrices held in 8-bit integers on tiles through
// LDS (slice_tile.hpp).
//
// C(m, n) = alpha sa(m) sb(n) sum_k a(m, k) b(n, k) + beta C(m, n), on
// v_mfma_i32_32x32x32_i8: 32 rows of A by 32 rows of B over 32 k, lane half h
// supplying 16 codes of row l % 32 of each operand.  A slice is 128 k: half h has
// its chunks 4 h .. 4 h + 3 and instruction s the s-th of them (which k an
// instruction adds does not matter, as long as A and B agree).
//
// Sums of whole numbers are exact, so that any tile gives the same bits.  8192^3 with a
// cast A: 430 to 476 us a product, by the card (2.3 to 2.55 POPS; a library product of
// 8-bit integers 465), the matrix cores 70% busy at the clock that power leaves them,
// after 40 to 47 us for the cast of A.  32 groups, 48 rows by 4096 x 2048: 37 us (5.2 TB/s of B's codes), and 5 for the cast.
#include "grouped_map.hpp"
#include "int8.hpp"
#include "slice_tile.hpp"

namespace sgemm {

namespace {

struct Int8Format {
  typedef i32x16 Acc;
  typedef slice_i32x4 Frag;
  static constexpr int kSteps = 4, kReads = 1, kMfma = 1, kChains = 2;
  template <int S, class At>
  __device__ __forceinline__ static Frag load(int half, At at) {
    return *at(4 * half + S);
  }
  template <int I>
  __device__ __forceinline__ static void mma(const Frag &a, const Frag &b, Acc &c) {
    c = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
};

template <int BM, int BN, int WM, int WN, int NST, bool CBF16>
__global__ void __launch_bounds__(WM *WN *kWave, 2)
int8_tile_kernel(Int8Args p, TileMap tmap, GroupMap map) {
  using Tile = SliceTile<Int8Format, BM, BN, WM, WN, NST>;
  constexpr int FM = Tile::FM, FN = Tile::FN;
  const int lane = threadIdx.x % kWave, r32 = lane % 32, half = lane / 32;

  long a_row = 0, b_row = 0;  // first row of the group in A (and C), and of its B
  int m0, n0, m_end = p.M;
  if (p.offsets) {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, BM, map);
    if (!t.valid) return;
    a_row = t.row0;
    b_row = (long)t.g * p.N;
    m0 = t.tm * BM;
    n0 = t.tn * BN;
    m_end = t.rows;
  } else {
    int bidx, tm, tn;
    tmap.tile(xcd_contiguous_id(blockIdx.x, gridDim.x), bidx, tm, tn);
    m0 = tm * BM;
    n0 = tn * BN;
  }
  const int rows_a = min(BM, m_end - m0), rows_b = min(BN, p.N - n0);
  // The tile's scales go to LDS while the first slices are on their way: read from
  // memory in the epilogue, each block of four rows waited for its own (17 us a
  // round of 256 x 256 tiles without stores, and without any k to speak of).
  const bool sums = p.K > 0;  // without k there are no scales either
  __shared__ __attribute__((aligned(16))) float scales_a[BM], scales_b[BN];
  for (int i = threadIdx.x; i < BM + BN; i += Tile::kThreads) {
    if (i < BM)
      scales_a[i] = sums && i < rows_a ? p.a.scales[a_row + m0 + i] : 0.f;
    else
      scales_b[i - BM] = sums && i - BM < rows_b ? p.b.scales[b_row + n0 + i - BM] : 0.f;
  }
  i32x16 acc[FM][FN];
  char *lds[NST];
  Tile::run(p.a.tile_rows(a_row + m0, rows_a), p.b.tile_rows(b_row + n0, rows_b),
            (p.K + 127) / 128, acc, lds);
  // run's barriers lie between the writes above and the reads below, but for K == 0,
  // where scales are not read.

  // Register e of lane l holds row acc32_row(l, e), column l % 32 of a block:
  // row 4 (l / 32) of a uniform base and a constant number of rows past it.
  using T = std::conditional_t<CBF16, __bf16, float>;
  const int mt = Tile::row0() + 4 * half, nt = Tile::col0() + r32;  // inside the tile
  T *const C = static_cast<T *>(p.C) + (a_row + m0 + Tile::row0()) * p.ldc + n0 + Tile::col0();
  const unsigned lane_at = (unsigned)((4 * half * p.ldc + r32) * sizeof(T));
  const int rows = rows_a - mt, cols = rows_b - nt;
  float scale_b[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) scale_b[j] = sums ? scales_b[nt + j * 32] : 0.f;
  auto store = [&](auto whole, auto with_c) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int quad = 0; quad < 4; ++quad) {
        const int r0 = i * 32 + 8 * quad;
        f32x4 scale_a = {0.f, 0.f, 0.f, 0.f};
        if (sums) scale_a = *reinterpret_cast<const f32x4 *>(scales_a + mt + r0);
        auto at = [&](int e, int j) {
          return reinterpret_cast<T *>(reinterpret_cast<char *>(C + (r0 + e) * p.ldc + j * 32) +
                                       lane_at);
        };
        auto in = [&](int e, int j) {
          return decltype(whole)::value || (r0 + e < rows && j * 32 < cols);
        };
        float c[4][FN];
        if constexpr (decltype(with_c)::value) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < FN; ++j) c[e][j] = in(e, j) ? (float)*at(e, j) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const float v = int8_value(acc[i][j][4 * quad + e], scale_a[e], scale_b[j]);
            if (!in(e, j)) continue;
            if constexpr (decltype(with_c)::value)
              *at(e, j) = (T)fmaf(p.alpha, v, p.beta * c[e][j]);
            else
              *at(e, j) = (T)(p.alpha * v);
          }
      }
  };
  const bool full = rows_a == BM && rows_b == BN;
  if (p.beta != 0.f)
    store(std::false_type(), std::true_type());
  else if (full)
    store(std::true_type(), std::false_type());
  else
    store(std::false_type(), std::false_type());
}

template <int BM, int BN, int WM, int WN, int NST>
hipError_t launch(const Int8Args &p, bool c_bf16, hipStream_t s) {
  const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  const long rows = p.offsets ? group_tile_rows(p.M, p.groups, BM) : tiles_m;
  const dim3 grid((unsigned)(rows * tiles_n)), block(WM * WN * kWave);
  const TileMap tmap = make_tile_map(tiles_m, tiles_n, kGroupRaster);
  const GroupMap map = make_group_map(tiles_n);
  if (c_bf16)
    hipLaunchKernelGGL((int8_tile_kernel<BM, BN, WM, WN, NST, true>), grid, block, 0, s, p, tmap,
                       map);
  else
    hipLaunchKernelGGL((int8_tile_kernel<BM, BN, WM, WN, NST, false>), grid, block, 0, s, p, tmap,
                       map);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_tile(const Int8Args &p, bool c_bf16, int cus, hipStream_t s) {
  switch (int8_tile(p, cus)) {
    case Int8Tile::k64_2: return launch<64, 64, 2, 2, 2>(p, c_bf16, s);
    case Int8Tile::k64_3: return launch<64, 64, 2, 2, 3>(p, c_bf16, s);
    case Int8Tile::k64_4: return launch<64, 64, 2, 2, 4>(p, c_bf16, s);
    case Int8Tile::k128: return launch<128, 128, 2, 4, 4>(p, c_bf16, s);
    case Int8Tile::k128x256: return launch<128, 256, 2, 4, 3>(p, c_bf16, s);
    default: return launch<256, 256, 2, 4, 2>(p, c_bf16, s);
  }
}

}  // namespace sgemm
