// mxfp4_gemm.hip -- products of few rows, or few rows a group, with a matrix
// held in microscaled 4-bit floating point (include/sgemm_mxfp4.h), and the
// choice between this kernel and the tiles of mxfp4_tile.hip.
//
// C(m, n) = alpha sum_b 2^(sa(m, b) + sb(n, b) - 254) sum_{k in b} a(m, k) b(n, k)
// + beta C(m, n) over blocks b of 32 k, on v_mfma_scale_f32_16x16x128_f8f6f4.
// The instruction multiplies 16 rows of A by 16 rows of B over 128 k; lane
// quarter q supplies one block of 32 codes (16 bytes) of row l % 16 of each
// operand, and that block's scale byte, which op_sel picks from the four bytes
// of a register.
//
// With few rows the time is that of reading B once, so B goes straight from
// global memory into registers, and k is split over the waves of a work-group
// to have enough of it in flight.  The four blocks that an instruction covers
// need not be neighbours, as long as A and B agree.  In a unit of 512 k (four
// granules of 128), quarter q has granule q and instruction s its block s: a
// lane then reads 64 consecutive bytes of codes and one dword of scales for
// four instructions, and the scales of 16 rows are 64 consecutive bytes.
//
// A of single precision or bfloat16 is cast by each wave as it needs it, a row
// of a unit at a time: 8 values a lane, so 4 lanes have a block and 16 a
// granule, as in the cast's own kernel.  The codes pass through LDS to the lanes
// that multiply them.  That costs each work-group the cast of its rows again,
// but no second launch: for one row by 8192 x 2048 it saves the cast's own 3
// us, as long as the product takes.
#include "grouped_map.hpp"
#include "mfma_dma.hpp"
#include "mxfp4.hpp"
#include "sgemm_mxfp4.h"

namespace sgemm {

namespace {

// All of A's rows (GROUPED: up to 16 MT of a group's), MT blocks of 16, and NT
// blocks of 16 rows of B per work-group; KS waves split k in units of 512.
// TA: A's type (SGEMM_TYPE_*).
template <int MT, int NT, int KS, int TA, bool CBF16, bool GROUPED>
__global__ void __launch_bounds__(KS *kWave) mxfp4_kernel(Mxfp4Args p, GroupMap map) {
  static_assert(TA == SGEMM_TYPE_MXFP4 || MT == 1, "only 16 rows are cast on the way");
  const int lane = threadIdx.x % kWave;
  const int kq = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r16 = lane % 16, q = lane / 16;
  const int granules = (p.K + 127) / 128;
  long a_row = 0, b_row = 0;  // first rows of A (and C) and of B
  int n0 = blockIdx.x * NT * 16, M = p.M;
  if constexpr (GROUPED) {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, 16 * MT, map);
    if (!t.valid) return;
    a_row = t.row0 + t.tm * (16 * MT);
    b_row = (long)t.g * p.N;
    n0 = t.tn * NT * 16;
    M = min(t.rows - t.tm * (16 * MT), 16 * MT);
  }

  // Rows past the end repeat the last one: what they give is not stored.
  const i32x4 *a_at[MT], *b_at[NT];
  const unsigned *as_at[MT], *bs_at[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long r = a_row + min(16 * i + r16, M - 1);
    a_at[i] = reinterpret_cast<const i32x4 *>(p.a.codes) + r * granules * 4;
    as_at[i] = p.a.scales + r;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const long r = b_row + min(n0 + 16 * j + r16, p.N - 1);
    b_at[j] = reinterpret_cast<const i32x4 *>(p.b.codes) + r * granules * 4;
    bs_at[j] = p.b.scales + r;
  }
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The cast A of one unit per wave: rows of 256 bytes of codes, 272 apart so
  // that 16 lanes' reads of a chunk fall on distinct banks, and their scales.
  constexpr int kPitch = 272 / 4;
  __shared__ __attribute__((aligned(16))) unsigned cast_codes[TA == SGEMM_TYPE_MXFP4 ? 4 : KS * 16 * kPitch];
  __shared__ unsigned cast_scales[TA == SGEMM_TYPE_MXFP4 ? 1 : KS * 16 * 4];

  struct Operand {
    i32x4 a[MT][4], b[NT][4];
    int as[MT], bs[NT];
  };
  // Granules past the last one give zeros.
  auto load = [&](int g0, Operand &o, auto whole) {
    const int g = g0 + q;
    const bool in = decltype(whole)::value || g < granules;
    const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int s = 0; s < 4; ++s) o.b[j][s] = in ? b_at[j][g * 4 + s] : zero;
      o.bs[j] = in ? (int)bs_at[j][g * p.b.lds] : 0;
    }
    if constexpr (TA == SGEMM_TYPE_MXFP4) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int s = 0; s < 4; ++s) o.a[i][s] = in ? a_at[i][g * 4 + s] : zero;
        o.as[i] = in ? (int)as_at[i][g * p.a.lds] : 0;
      }
    }
  };
  auto cast = [&](int g0, Operand &o) {
    constexpr bool BF16 = TA == SGEMM_TYPE_BF16;
    unsigned *codes = cast_codes + kq * 16 * kPitch, *scales = cast_scales + kq * 16 * 4;
    const int k = g0 * 128 + lane * 8;
    const long row_bytes = p.a.lds * (BF16 ? 2 : 4);
    const char *x = reinterpret_cast<const char *>(p.a.codes) + a_row * row_bytes +
                    (long)k * (BF16 ? 2 : 4);
    for (int r = 0; r < M; r += 4) {  // four rows' loads go out together
      float v[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) load8<BF16>(x + min(r + i, M - 1) * row_bytes, p.K - k, v[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r + i >= M) break;
        unsigned all;
        codes[(r + i) * kPitch + lane] = mxfp4_cast8(v[i], lane, all);
        if (r16 == 0) scales[(r + i) * 4 + q] = all;
      }
    }
    // The wave's own LDS accesses keep their order; the fence keeps the
    // compiler's.
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int r = min(r16, M - 1);
#pragma unroll
    for (int s = 0; s < 4; ++s)
      o.a[0][s] = *reinterpret_cast<const i32x4 *>(codes + r * kPitch + q * 16 + s * 4);
    o.as[0] = (int)scales[r * 4 + q];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  auto mma = [&](const Operand &o) {
    static_for<4>([&](auto S) {
      constexpr int s = decltype(S)::value;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = mfma_fp4_16x16x128<s>(o.a[i][s], o.b[j][s], acc[i][j], o.as[i], o.bs[j]);
    });
  };
  auto load_any = [&](int g0, Operand &o) {
    if (g0 + 4 <= granules)
      load(g0, o, std::true_type());
    else if (g0 < granules)
      load(g0, o, std::false_type());
  };
  // The next unit's B (and held A) is on its way while this one is multiplied.
  Operand cur, nxt;
  load_any(4 * kq, cur);
  for (int g0 = 4 * kq; g0 < granules; g0 += 4 * KS) {
    load_any(g0 + 4 * KS, nxt);
    if constexpr (TA != SGEMM_TYPE_MXFP4) cast(g0, cur);
    mma(cur);
    cur = nxt;
  }

  __shared__ f32x4 red[(KS - 1) * MT * NT * kWave];
  if (kq > 0) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        red[((kq - 1) * MT * NT + i * NT + j) * kWave + lane] = acc[i][j];
  }
  __syncthreads();
  if (kq > 0) return;
#pragma unroll
  for (int s = 0; s < KS - 1; ++s)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] += red[(s * MT * NT + i * NT + j) * kWave + lane];

  // Register e of lane l holds row 4 (l / 16) + e, column l % 16 of a block.
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = 16 * i + 4 * q + e;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int n = n0 + 16 * j + r16;
        if (n >= p.N) continue;
        store_c<CBF16>(p, (a_row + m) * p.ldc + n, acc[i][j][e]);
      }
    }
}

template <int MT, int NT, int KS, int TA, bool GROUPED>
hipError_t launch_sets(const Mxfp4Args &p, bool c_bf16, hipStream_t s) {
  const int tiles_n = (int)((p.N + NT * 16L - 1) / (NT * 16));
  const long rows = GROUPED ? group_tile_rows(p.M, p.groups, 16 * MT) : 1;
  const dim3 grid((unsigned)(rows * tiles_n)), block(KS * kWave);
  const GroupMap map = make_group_map(tiles_n);
  if (c_bf16)
    hipLaunchKernelGGL((mxfp4_kernel<MT, NT, KS, TA, true, GROUPED>), grid, block, 0, s, p, map);
  else
    hipLaunchKernelGGL((mxfp4_kernel<MT, NT, KS, TA, false, GROUPED>), grid, block, 0, s, p, map);
  return hipGetLastError();
}

template <int MT, int NT, int TA>
hipError_t launch(const Mxfp4Args &p, bool c_bf16, hipStream_t s) {
  return mxfp4_eight_sets(p.K) ? launch_sets<MT, NT, 8, TA, false>(p, c_bf16, s)
                               : launch_sets<MT, NT, 4, TA, false>(p, c_bf16, s);
}

template <int TA>
hipError_t launch_rows(const Mxfp4Args &p, bool c_bf16, hipStream_t s) {
  return p.offsets ? launch_sets<1, 1, 4, TA, true>(p, c_bf16, s)
                   : launch<1, 1, TA>(p, c_bf16, s);
}

// Rows spread thin over groups, in few work-groups (16 columns each; the host
// counts a row of tiles for each group that can have rows).  Measured with A of
// bfloat16, the cast and the 64 x 64 tile first: 64 groups, 8 rows by 2048 x
// 2048 11.3 us and 8.1; 128 groups, 8 rows by 768 x 2048 10.6 and 6.4; 16 groups,
// 24 rows by 2048 x 2048 14.9 and 12.4; 8 groups, 16 rows by 4096 x 4096 21.5 and
// 21.6, 64 rows 21.5 and 41.7; 32 groups, 48 rows by 4096 x 2048 31.5 and 38.2.
// A held: 64 groups, 8 rows by 2048 x 2048 8.5 and 6.9.
bool spread_thin(const Mxfp4Args &p, int cus) {
  const long groups = p.groups < p.M ? p.groups : p.M;
  return p.M <= 2L * p.groups && groups * ((p.N + 15L) / 16) <= 8L * cus;
}

}  // namespace

// Casting M rows in every work-group beats a launch of the cast while the
// rows are short and few: 1 x 8192 x 2048 4.8 us against 2.7 + 4.0, 2 x 8192 x
// 8192 11.9 against 2.8 + 9.9; 4 x 8192 x 8192 13.9 against 2.6 + 10.2.
bool mxfp4_casts(const Mxfp4Args &p, int cus) {
  if (p.offsets) return spread_thin(p, cus);
  return p.M <= 16 && (long)p.M * p.K <= 16384;
}

// Up to 32 rows, and rows spread thin over groups, this kernel: 16 x 8192 x 8192
// 12.3 us (64 x 64 tile 18.2), 32 rows 14.3 (18.5); 64 rows 21.4 (19.2).
hipError_t launch_mxfp4_product(const Mxfp4Args &p, int a_type, bool c_bf16, int cus,
                                hipStream_t s) {
  if (a_type == SGEMM_TYPE_F32) return launch_rows<SGEMM_TYPE_F32>(p, c_bf16, s);
  if (a_type == SGEMM_TYPE_BF16) return launch_rows<SGEMM_TYPE_BF16>(p, c_bf16, s);
  if (p.offsets ? !spread_thin(p, cus) : p.M > 32) return launch_mxfp4_tile(p, c_bf16, cus, s);
  return p.offsets || p.M <= 16 ? launch_rows<SGEMM_TYPE_MXFP4>(p, c_bf16, s)
                                : launch<2, 2, SGEMM_TYPE_MXFP4>(p, c_bf16, s);
}

}  // namespace sgemm
