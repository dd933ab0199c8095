// grouped.hip -- single-precision products of short groups of rows
// (include/sgemm_grouped.h), and the choice between this kernel and the tiles
// of grouped_tile.hip.
//
// C(r, :) = alpha sum_k A(r, k) op(B_g)(k, :) + beta C(r, :) for the rows r of
// group g, on v_mfma_f32_16x16x4_f32.  With a few rows a group the time is that
// of reading the B_g once.  A work-group has 16 rows by 64 columns and splits k
// over four waves, whose sums are added in order at the end, so that even one
// short group spreads over the chip; its operands go straight from global
// memory into registers.
//
// K is walked in groups of 16; in one, lane quarter h supplies k = 4 h + t to
// instruction t, so an operand whose k runs along its stored rows takes its
// four instructions' values in one 16-byte load.  B as given takes four 16-byte
// loads, one of each k row, and its 64 columns are dealt to the four blocks
// in turn: block j has column 4 c + j of lane c.
//
// 24 rows in 16 groups by 2048 x 2048: 31.5 us, 6.4 TB/s of the weights that
// have rows (part of them stays in the Infinity Cache between calls).
#include <type_traits>

#include "common.hpp"
#include "grouped.hpp"
#include "grouped_map.hpp"

namespace sgemm {

namespace {

// Four floats at any 4-byte aligned address.
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

// The first n (0..4) of four consecutive floats, zeros for the others.
__device__ __forceinline__ f32x4 load_some(const float *p, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    v = *reinterpret_cast<const f32x4_u *>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) v[e] = p[e];
  }
  return v;
}

constexpr int kRows = 16, kCols = 64, kSets = 4;

template <bool TB>
__global__ void __launch_bounds__(kSets *kWave) grouped_kernel(GroupedArgs p, GroupMap map) {
  const int lane = threadIdx.x % kWave;
  const int kq = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, h = lane / 16;

  const GroupTile t = group_tile(p.offsets, p.groups, p.M, kRows, map);
  if (!t.valid) return;
  const float *A = p.A + t.row0 * p.lda, *B = p.B + (long)t.g * p.strideB;
  float *C = p.C + t.row0 * p.ldc;
  const int K = p.alpha != 0.f ? p.K : 0;
  const float alpha = K > 0 ? p.alpha : 0.f;  // an empty sum is 0, whatever alpha is
  const int m0 = t.tm * kRows, n0 = t.tn * kCols, m_end = t.rows;

  struct Ops {
    f32x4 a, b[4];
  };
  // Rows past the end repeat the last one: what they give is not stored.
  const float *const a_row = A + (long)min(m0 + c, m_end - 1) * p.lda;
  auto load = [&](int k, Ops &o, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    o.a = load_some(a_row + k + 4 * h, WHOLE ? 4 : K - k - 4 * h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TB) {
        const int n = min(n0 + 16 * j + c, p.N - 1), kk = k + 4 * h;
        o.b[j] = load_some(B + (long)n * p.ldb + kk, WHOLE ? 4 : K - kk);
      } else {
        const int kk = k + 4 * h + j, n = n0 + 4 * c;
        o.b[j] = load_some(B + (long)kk * p.ldb + n, WHOLE ? 4 : (kk < K ? p.N - n : 0));
      }
    }
  };
  f32x4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bool inside = TB || n0 + kCols <= p.N;
  for (int k = 16 * kq; k < K; k += 16 * kSets) {
    Ops o;
    if (inside && k + 16 <= K)
      load(k, o, std::true_type());
    else
      load(k, o, std::false_type());
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j] = mfma16x16x4(o.a[t], TB ? o.b[j][t] : o.b[t][j], acc[j]);
  }

  __shared__ f32x4 red[(kSets - 1) * 4 * kWave];
  if (kq > 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) red[((kq - 1) * 4 + j) * kWave + lane] = acc[j];
  }
  __syncthreads();
  if (kq > 0) return;
#pragma unroll
  for (int s = 0; s < kSets - 1; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += red[(s * 4 + j) * kWave + lane];

  // Register e of lane l holds row 4 (l / 16) + e, column l % 16 of a block.
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int m = m0 + 4 * h + e;
    if (m >= m_end) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = TB ? n0 + 16 * j + c : n0 + 4 * c + j;
      if (n >= p.N) continue;
      float *at = C + (long)m * p.ldc + n;
      *at = p.beta == 0.f ? alpha * acc[j][e] : fmaf(alpha, acc[j][e], p.beta * *at);
    }
  }
}

}  // namespace

// This kernel or a tile of 32 x 128 through LDS, whichever the rounds of
// work-groups on the compute units make faster.  A round of the tile takes as
// long as 2.4 rounds of this kernel, 1.6 where B is transposed or its loads are
// narrow.  Measured, this kernel first: 1 group of 64 rows by 4096 x 4096 42 us
// and 75; 16 groups, 24 rows by 2048 x 2048 31.5 and 42.5, 512 rows 61 and 67,
// 1024 rows 108 and 102; 64 groups, 2048 rows by 1024 x 1024 63 and 45; B
// transposed 16 groups, 384 rows by 2048 x 2048 96 and 79.  The host knows the
// number of tiles to within the groups' lengths.
hipError_t launch_grouped_rows(const GroupedArgs &p, bool tb, int cus, hipStream_t s) {
  const long groups = p.groups < p.M ? p.groups : p.M;
  auto rounds = [&](long bm, long bn) {
    const long most = p.M / bm + groups / 2;
    return ((most > groups ? most : groups) * ((p.N + bn - 1) / bn) + cus - 1) / cus;
  };
  const double per_round = tb || p.N % 4 != 0 ? 0.625 : 0.42;
  if (rounds(kRows, kCols) * per_round > rounds(32, 128))
    return launch_grouped_tile(p, tb, cus, s);
  const int tiles_n = (p.N + kCols - 1) / kCols;
  const dim3 grid((unsigned)(group_tile_rows(p.M, p.groups, kRows) * tiles_n)),
      block(kSets * kWave);
  if (tb)
    hipLaunchKernelGGL(grouped_kernel<true>, grid, block, 0, s, p, make_group_map(tiles_n));
  else
    hipLaunchKernelGGL(grouped_kernel<false>, grid, block, 0, s, p, make_group_map(tiles_n));
  return hipGetLastError();
}

}  // namespace sgemm
