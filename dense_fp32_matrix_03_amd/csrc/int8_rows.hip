// int8_rows.hip -- products of few rows, or few rows a group, with a matrix held in
// 8-bit integers (include/sgemm_int8.h), and the launch of this kernel or of the tiles of
// int8_tile.hip.
//
// C(m, n) = alpha sa(m) sb(n) sum_k a(m, k) b(n, k) + beta C(m, n), on
// v_mfma_i32_16x16x64_i8: 16 rows of A by 16 rows of B over 64 k, lane quarter q
// supplying 16 codes of row l % 16 of each operand.
//
// With few rows the time is that of reading B once, so B goes straight from
// global memory into registers, and k is split over the waves of a work-group to
// have enough of it in flight.  Which k an instruction adds does not matter, as long
// as A and B agree: in a unit of 256 k, quarter q has k 64 q .. 64 q + 63 and
// instruction s the s-th 16 of them, so that a lane reads 64 consecutive bytes.
//
// A of single precision or bfloat16 is cast by each work-group as it needs it,
// without a launch for the cast: every wave finds its share's largest magnitudes
// while its first codes of B are on their way, the work-group's waves exchange
// them, and then each casts the k that it multiplies, 4 values a lane; the codes
// pass through LDS to the lanes that multiply them.
//
// 1 x 8192 x 2048 from bfloat16: 6.1 us by graph replay, of which reading B takes 3.4 at a
// large copy's rate; the rest is the launch, and x, its largest magnitude and the codes
// one after the other.
#include "grouped_map.hpp"
#include "int8.hpp"
#include "mfma_dma.hpp"
#include "sgemm_int8.h"

namespace sgemm {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// All of A's rows, 16 at most (GROUPED: 16 of a group's), and 16 rows of B per
// work-group; KS waves split k in units of 256.  TA: A's type (SGEMM_TYPE_*).
template <int KS, int TA, bool CBF16, bool GROUPED>
__global__ void __launch_bounds__(KS *kWave) int8_rows_kernel(Int8Args p, GroupMap map) {
  constexpr bool CAST = TA != SGEMM_TYPE_INT8;
  constexpr int kUnit = 256;
  const int lane = threadIdx.x % kWave;
  const int kq = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r16 = lane % 16, q = lane / 16;
  const int kp = (p.K + 127) / 128 * 128;
  long a_row = 0, b_row = 0;  // first rows of A (and C) and of B
  int n0 = blockIdx.x * 16, M = p.M;
  if constexpr (GROUPED) {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, 16, map);
    if (!t.valid) return;
    a_row = t.row0 + t.tm * 16;
    b_row = (long)t.g * p.N;
    n0 = t.tn * 16;
    M = min(t.rows - t.tm * 16, 16);
  }

  // Rows past the end repeat the last one: what they give is not stored.
  const char *const a_at = p.a.codes + (a_row + min(r16, M - 1)) * p.a.ld;
  const long b_at_row = b_row + min(n0 + r16, p.N - 1);
  const char *const b_at = p.b.codes + b_at_row * p.b.ld + 64 * q;
  const float scale_b = p.K > 0 ? p.b.scales[b_at_row] : 0.f;
  i32x4 acc = {0, 0, 0, 0};

  struct Operand {
    i32x4 a[4], b[4];
  };
  // Quarters past the padded k give zeros.
  auto load = [&](int k, Operand &o, auto whole) {
    const bool in = decltype(whole)::value || k + 64 * q < kp;
    const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      o.b[s] = in ? *reinterpret_cast<const i32x4 *>(b_at + k + 16 * s) : zero;
    if constexpr (!CAST) {
      const char *const at = a_at + (k / 128 + q / 2) * p.a.slice + 64 * (q % 2);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        o.a[s] = in ? *reinterpret_cast<const i32x4 *>(at + 16 * s) : zero;
    }
  };
  auto load_any = [&](int k, Operand &o) {
    if (k + kUnit <= kp)
      load(k, o, std::true_type());
    else if (k < kp)
      load(k, o, std::false_type());
  };
  Operand cur, nxt;
  load_any(kUnit * kq, cur);

  // The cast A of one unit per wave: rows of 256 bytes of codes, 272 apart so
  // that 16 lanes' reads of a chunk fall on distinct banks.
  constexpr int kPitch = 272 / 4;
  __shared__ __attribute__((aligned(16))) unsigned cast_codes[CAST ? KS * 16 * kPitch : 4];
  __shared__ unsigned tops[CAST ? KS : 1][16];
  __shared__ float scales[16], inverses[16];
  constexpr bool BF16 = TA == SGEMM_TYPE_BF16;
  const long row_bytes = p.a.ld * (BF16 ? 2 : 4);
  const char *const x = p.a.codes + a_row * row_bytes;
  // Values 4 lane .. + 3 of a unit, zeros past K.
  auto values = [&](int row, int k, float v[4]) {
    k += 4 * lane;
    const char *at = x + row * row_bytes + (long)k * (BF16 ? 2 : 4);
    if (k + 4 <= p.K) {
      if constexpr (BF16) {
        typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
        const u32x2_any t = *reinterpret_cast<const u32x2_any *>(at);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[2 * e] = __uint_as_float(t[e] << 16);
          v[2 * e + 1] = __uint_as_float(t[e] & 0xffff0000u);
        }
      } else {
        const f32x4_any t = *reinterpret_cast<const f32x4_any *>(at);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = t[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = 0.f;
        if (k + e >= p.K) continue;
        if constexpr (BF16)
          v[e] = __uint_as_float((unsigned)reinterpret_cast<const unsigned short *>(at)[e] << 16);
        else
          v[e] = reinterpret_cast<const float *>(at)[e];
      }
    }
  };
  if constexpr (CAST) {
    for (int r = 0; r < M; ++r) {
      unsigned top = 0;
      for (int k = kUnit * kq; k < p.K; k += kUnit * KS) {
        float v[4];
        values(r, k, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
      }
#pragma unroll
      for (int d = 32; d > 0; d /= 2) top = max(top, (unsigned)__shfl_xor((int)top, d));
      if (lane == 0) tops[kq][r] = top;
    }
    __syncthreads();
    if (threadIdx.x < 16 && threadIdx.x < M) {
      unsigned top = 0;
#pragma unroll
      for (int w = 0; w < KS; ++w) top = max(top, tops[w][threadIdx.x]);
      const Int8Scale s(int8_scale(top));
      scales[threadIdx.x] = s.scale;
      inverses[threadIdx.x] = s.inverse;
    }
    __syncthreads();
  }
  auto cast = [&](int k, Operand &o) {
    unsigned *codes = cast_codes + kq * 16 * kPitch;
    for (int r = 0; r < M; ++r) {
      const Int8Scale s(scales[r], inverses[r]);
      float v[4];
      values(r, k, v);
      int8_codes<4>(s, v, codes + r * kPitch + lane);
    }
    // The wave's own LDS accesses keep their order; the fence keeps the
    // compiler's.
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int r = min(r16, M - 1);
#pragma unroll
    for (int s = 0; s < 4; ++s)
      o.a[s] = *reinterpret_cast<const i32x4 *>(codes + r * kPitch + q * 16 + s * 4);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  // The next unit's B (and held A) is on its way while this one is multiplied.
  for (int k = kUnit * kq; k < kp; k += kUnit * KS) {
    load_any(k + kUnit * KS, nxt);
    if constexpr (CAST) cast(k, cur);
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur.a[s], cur.b[s], acc, 0, 0, 0);
    cur = nxt;
  }

  __shared__ i32x4 red[(KS - 1) * kWave];
  if (kq > 0) red[(kq - 1) * kWave + lane] = acc;
  __syncthreads();
  if (kq > 0) return;
#pragma unroll
  for (int s = 0; s < KS - 1; ++s) acc += red[s * kWave + lane];

  // Register e of lane l holds row 4 (l / 16) + e, column l % 16 of the block.
  using T = std::conditional_t<CBF16, __bf16, float>;
  const int n = n0 + r16;
  if (n >= p.N) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int m = 4 * q + e;
    if (m >= M) continue;
    float sa = 0.f;
    if (p.K > 0) sa = CAST ? scales[m] : p.a.scales[a_row + m];
    T *const C = static_cast<T *>(p.C) + (a_row + m) * p.ldc + n;
    const float v = int8_value(acc[e], sa, scale_b);
    *C = (T)(p.beta == 0.f ? p.alpha * v : fmaf(p.alpha, v, p.beta * (float)*C));
  }
}

template <int KS, int TA, bool GROUPED>
hipError_t launch(const Int8Args &p, bool c_bf16, hipStream_t s) {
  const int tiles_n = (int)((p.N + 15L) / 16);
  const long rows = GROUPED ? group_tile_rows(p.M, p.groups, 16) : 1;
  const dim3 grid((unsigned)(rows * tiles_n)), block(KS * kWave);
  const GroupMap map = make_group_map(tiles_n);
  if (c_bf16)
    hipLaunchKernelGGL((int8_rows_kernel<KS, TA, true, GROUPED>), grid, block, 0, s, p, map);
  else
    hipLaunchKernelGGL((int8_rows_kernel<KS, TA, false, GROUPED>), grid, block, 0, s, p, map);
  return hipGetLastError();
}

// Eight waves where there are more than four units of k.
template <int TA>
hipError_t launch_rows(const Int8Args &p, bool c_bf16, hipStream_t s) {
  if (p.offsets) return launch<4, TA, true>(p, c_bf16, s);
  return p.K > 1024 ? launch<8, TA, false>(p, c_bf16, s) : launch<4, TA, false>(p, c_bf16, s);
}

}  // namespace

// Casting a row in every work-group beats a launch of the cast while the values are few
// and a wave has a single unit of k: 1 x 8192 x 2048 7.2 us against 10.5, 4 x 8192 x 2048
// 9.1 against 10.8, 8 x 4096 x 1024 8.3 against 9.2; 8 x 8192 x 2048 12.5 against 10.4, 2
// x 14336 x 4096 22.4 against 17.8.  In groups, a row each: 64 groups, 8 rows by 2048 x
// 2048 10.9 against 13.8; 16 groups, 24 rows by 2048 x 2048 21.2 against 14.7.
bool int8_casts(const Int8Args &p, int cus) {
  if (p.K > 2048) return false;
  if (p.offsets)
    return int8_spread_thin(p, cus) && p.M <= p.groups && (long)p.M * p.K <= 16384;
  return p.M <= 16 && (long)p.M * p.K <= 8192;
}

hipError_t launch_int8_product(const Int8Args &p, int a_type, bool c_bf16, int cus, hipStream_t s) {
  if (a_type == SGEMM_TYPE_F32) return launch_rows<SGEMM_TYPE_F32>(p, c_bf16, s);
  if (a_type == SGEMM_TYPE_BF16) return launch_rows<SGEMM_TYPE_BF16>(p, c_bf16, s);
  return int8_few_rows(p, cus) ? launch_rows<SGEMM_TYPE_INT8>(p, c_bf16, s)
                               : launch_int8_tile(p, c_bf16, cus, s);
}

}  // namespace sgemm
