// grouped.hip -- single-precision products whose rows fall into groups of
// unequal length (include/sgemm_grouped.h).
//
// C(r, :) = alpha sum_k A(r, k) op(B_g)(k, :) + beta C(r, :) for the rows r of
// group g, and C_g = alpha sum_r A(r, :)^T B(r, :) + beta C_g.  Both sum
// products of FP32 values on v_mfma_f32_16x16x4_f32.
//
// Operands go straight from global memory into registers.  K is walked in
// groups of 16; in one, lane quarter h supplies k = 4 h + t to instruction t,
// so an operand whose k runs along its stored rows takes its four
// instructions' values in one 16-byte load.  An operand stored the other way
// takes four 16-byte loads, one of each k row, and its 64 rows (or columns)
// are dealt to the four blocks in turn: block j has 4 c + j of lane c.
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

// Where the operands' k runs.
enum Layout { kNN, kNT, kTN };  // B as given; B transposed; A transposed (grouped_k)

// MT: blocks of 16 rows per wave; a wave has 64 columns.  WM x WN waves share
// a tile, each with KS waves that split k between them (16 k in turn).
template <int LAYOUT, int MT, int WM, int WN, int KS>
__global__ void __launch_bounds__(WM *WN *KS *kWave) grouped_kernel(GroupedArgs p, int tiles_m,
                                                                   int tiles_n) {
  constexpr bool TA = LAYOUT == kTN, TB = LAYOUT == kNT;
  static_assert(!TA || MT == 4, "a transposed A gives blocks of 64 rows");
  constexpr int BM = WM * MT * 16, BN = WN * 64;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int kq = wave % KS, wm = wave / KS % WM, wn = wave / (KS * WM);
  const int c = lane % 16, h = lane / 16;

  const float *A = p.A, *B = p.B;
  float *C = p.C;
  int m0, n0, m_end, K;  // the wave's tile inside the group's rows, and its k
  if constexpr (TA) {
    const int per = tiles_m * tiles_n;
    const int g = blockIdx.x / per, t = blockIdx.x % per;
    long first, last;
    group_range(p.offsets, g, p.K, first, last);
    A += first * p.lda;
    B += first * p.ldb;
    C += (long)g * p.strideC;
    K = (int)(last - first);
    m0 = t / tiles_n * BM;
    n0 = t % tiles_n * BN;
    m_end = p.M;
  } else {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, BM, tiles_n, 8);
    if (!t.valid) return;
    A += t.row0 * p.lda;
    B += (long)t.g * p.strideB;
    C += t.row0 * p.ldc;
    K = p.K;
    m0 = t.tm * BM;
    n0 = t.tn * BN;
    m_end = t.rows;
  }
  m0 += wm * MT * 16;
  n0 += wn * 64;

  struct Ops {
    f32x4 a[4], b[4];
  };
  // Rows past the end repeat the last one: what they give is not stored.
  auto load = [&](int k, Ops &o, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    if constexpr (TA) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int kk = k + 4 * h + t, m = m0 + 4 * c;
        const float *at = A + (long)kk * p.lda + m;
        o.a[t] = load_some(at, WHOLE ? 4 : (kk < K ? m_end - m : 0));
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = min(m0 + 16 * i + c, m_end - 1), kk = k + 4 * h;
        o.a[i] = load_some(A + (long)m * p.lda + kk, WHOLE ? 4 : K - kk);
      }
    }
    if constexpr (TB) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = min(n0 + 16 * j + c, p.N - 1), kk = k + 4 * h;
        o.b[j] = load_some(B + (long)n * p.ldb + kk, WHOLE ? 4 : K - kk);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int kk = k + 4 * h + t, n = n0 + 4 * c;
        o.b[t] = load_some(B + (long)kk * p.ldb + n, WHOLE ? 4 : (kk < K ? p.N - n : 0));
      }
    }
  };
  f32x4 acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mma = [&](const Ops &o) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = mfma16x16x4(TA ? o.a[t][i] : o.a[i][t], TB ? o.b[j][t] : o.b[t][j],
                                  acc[i][j]);
  };

  if (p.alpha != 0.f && m0 < m_end && n0 < p.N) {
    const bool inside = (!TA || m0 + 64 <= m_end) && (TB || n0 + 64 <= p.N);
    for (int k = 16 * kq; k < K; k += 16 * KS) {
      Ops o;
      if (inside && k + 16 <= K)
        load(k, o, std::true_type());
      else
        load(k, o, std::false_type());
      mma(o);
    }
  }

  if constexpr (KS > 1) {
    __shared__ f32x4 red[WM * WN * (KS - 1) * MT * 4 * kWave];
    f32x4 *mine = red + (wm + wn * WM) * (KS - 1) * MT * 4 * kWave + lane;
    if (kq > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mine[((kq - 1) * MT * 4 + i * 4 + j) * kWave] = acc[i][j];
    }
    __syncthreads();
    if (kq > 0) return;
#pragma unroll
    for (int s = 0; s < KS - 1; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += mine[(s * MT * 4 + i * 4 + j) * kWave];
  }

  // Register e of lane l holds row 4 (l / 16) + e, column l % 16 of a block.
  const bool plain = p.alpha == 1.f && p.beta == 0.f;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * h + e;
      const int m = TA ? m0 + 4 * r + i : m0 + 16 * i + r;
      if (m >= m_end) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = TB ? n0 + 16 * j + c : n0 + 4 * c + j;
        if (n >= p.N) continue;
        float *at = C + (long)m * p.ldc + n;
        if (plain)
          *at = acc[i][j][e];
        else if (p.beta == 0.f)
          *at = p.alpha * acc[i][j][e];
        else
          *at = fmaf(p.alpha, acc[i][j][e], p.beta * *at);
      }
    }
}

}  // namespace

hipError_t launch_grouped_rows(const GroupedArgs &p, bool tb, int cus, hipStream_t s) {
  const int tiles_n = (p.N + 63) / 64;
  const dim3 grid((unsigned)(group_tile_rows(p.M, p.groups, 16) * tiles_n)), block(4 * kWave);
  if (tb)
    hipLaunchKernelGGL((grouped_kernel<kNT, 1, 1, 1, 4>), grid, block, 0, s, p, 0, tiles_n);
  else
    hipLaunchKernelGGL((grouped_kernel<kNN, 1, 1, 1, 4>), grid, block, 0, s, p, 0, tiles_n);
  return hipGetLastError();
}

hipError_t launch_grouped_k(const GroupedArgs &p, int cus, hipStream_t s) {
  const int tiles_m = (p.M + 127) / 128, tiles_n = (p.N + 127) / 128;
  const dim3 grid((unsigned)((long)tiles_m * tiles_n * p.groups)), block(4 * kWave);
  hipLaunchKernelGGL((grouped_kernel<kTN, 4, 2, 2, 1>), grid, block, 0, s, p, tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace sgemm
