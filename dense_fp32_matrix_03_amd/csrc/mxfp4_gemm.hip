// mxfp4_gemm.hip -- products of matrices held in microscaled 4-bit floating
// point (include/sgemm_mxfp4.h), on v_mfma_scale_f32_16x16x128_f8f6f4.
//
// C(m, n) = alpha sum_b 2^(sa(m, b) + sb(n, b) - 254) sum_{k in b} a(m, k) b(n, k)
// + beta C(m, n) over blocks b of 32 k.  The instruction multiplies 16 rows of
// A by 16 rows of B over 128 k; lane quarter q supplies one block of 32 codes
// (16 bytes) of row l % 16 of each operand, and that block's scale byte, which
// op_sel picks from the four bytes of a register.
//
// The four blocks that an instruction covers need not be neighbours, as long
// as A and B agree.  In a unit of 512 k (four granules of 128), quarter q has
// granule q and instruction s its block s: a lane then reads 64 consecutive
// bytes of codes and one dword of scales for four instructions, and the
// scales of 16 rows are 64 consecutive bytes.
#include "grouped_map.hpp"
#include "mxfp4.hpp"
#include "mfma_dma.hpp"

namespace sgemm {

namespace {

// MT x NT blocks of 16 x 16 per wave; KS waves split k in units of 512.
template <int MT, int NT, int KS, bool CBF16>
__global__ void __launch_bounds__(KS *kWave) mxfp4_kernel(Mxfp4Args p, int tiles_m, int tiles_n) {
  const int lane = threadIdx.x % kWave;
  const int kq = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r16 = lane % 16, q = lane / 16;
  const int granules = (p.K + 127) / 128;
  long a_row = 0, b_row = 0;  // first row of the group in A (and C), and of its B
  int m0, n0, m_end = p.M;
  if (p.offsets) {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, MT * 16, tiles_n, 8);
    if (!t.valid) return;
    a_row = t.row0;
    b_row = (long)t.g * p.N;
    m0 = t.tm * MT * 16;
    n0 = t.tn * NT * 16;
    m_end = t.rows;
  } else {
    m0 = (int)(blockIdx.x / tiles_n) * MT * 16;
    n0 = (int)(blockIdx.x % tiles_n) * NT * 16;
  }

  // Rows past the end repeat the last one: what they give is not stored.
  const i32x4 *a_at[MT], *b_at[NT];
  const unsigned *as_at[MT], *bs_at[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long r = a_row + min(m0 + 16 * i + r16, m_end - 1);
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

  const int nk = p.alpha != 0.f ? granules : 0;
  for (int g0 = 4 * kq; g0 < nk; g0 += 4 * KS) {
    const int g = g0 + q;
    const bool in = g < granules;
    i32x4 a[MT][4], b[NT][4];
    int as[MT], bs[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      as[i] = in ? (int)as_at[i][g * p.a.lds] : 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) a[i][s] = in ? a_at[i][g * 4 + s] : i32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      bs[j] = in ? (int)bs_at[j][g * p.b.lds] : 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) b[j][s] = in ? b_at[j][g * 4 + s] : i32x4{0, 0, 0, 0};
    }
    static_for<4>([&](auto S) {
      constexpr int s = decltype(S)::value;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = mfma_fp4_16x16x128<s>(a[i][s], b[j][s], acc[i][j], as[i], bs[j]);
    });
  }

  if constexpr (KS > 1) {
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
  }

  // Register e of lane l holds row 4 (l / 16) + e, column l % 16 of a block.
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = m0 + 16 * i + 4 * q + e;
      if (m >= m_end) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int n = n0 + 16 * j + r16;
        if (n >= p.N) continue;
        store_c<CBF16>(p, (a_row + m) * p.ldc + n, acc[i][j][e]);
      }
    }
}

// The tile through LDS.  In units of a 256 x 256 tile's time, a compute unit
// takes 0.56 for one tile of 128 x 128, 0.73 for two (they share it), and 0.29
// a tile for more: measured on 256 compute units with bfloat16 C, 2048^3 24.0
// us with 64 tiles of 256 x 256 and 13.5 with 256 of 128 x 128, 1024 x 8192 x
// 8192 56.3 (128 tiles) and 40.8 (512), 4096^3 38.8 (256) and 42.9 (1024),
// 8192^3 250 (1024) and 298 (4096).  Groups count with their mean length.
int mxfp4_tile_size(const Mxfp4Args &p, int cus) {
  const long groups = p.offsets ? p.groups : 1, mean = (p.M + groups - 1) / groups;
  auto per_cu = [&](long t) {
    const long tiles = groups * ((mean + t - 1) / t) * ((p.N + t - 1) / t);
    return (double)((tiles + cus - 1) / cus);
  };
  const double n = per_cu(128);
  return per_cu(256) <= (n == 1 ? 0.56 : n == 2 ? 0.73 : 0.29 * n) ? 256 : 128;
}

}  // namespace

hipError_t launch_mxfp4_product(const Mxfp4Args &p, bool c_bf16, int cus, hipStream_t s) {
  const long mean = p.M / (p.offsets ? p.groups : 1);
  if (mean > 64) return launch_mxfp4_tile(mxfp4_tile_size(p, cus), p, c_bf16, s);
  const int tiles_n = (p.N + 31) / 32, tiles_m = (p.M + 15) / 16;
  const long rows = p.offsets ? group_tile_rows(p.M, p.groups, 16) : tiles_m;
  const dim3 grid((unsigned)(rows * tiles_n)), block(4 * kWave);
  if (c_bf16)
    hipLaunchKernelGGL((mxfp4_kernel<1, 2, 4, true>), grid, block, 0, s, p, tiles_m, tiles_n);
  else
    hipLaunchKernelGGL((mxfp4_kernel<1, 2, 4, false>), grid, block, 0, s, p, tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace sgemm
