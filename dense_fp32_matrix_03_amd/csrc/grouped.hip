// grouped.hip -- single-precision products of grouped rows
// (include/sgemm_grouped.h) whose operand slices reach LDS by buffer-to-LDS
// loads: the pipeline, LDS images and k order of mfma_dma.hpp, with a tile's
// operands and limits found from the group lengths on the device.
//
// C(r, :) = alpha sum_k A(r, k) op(B_g)(k, :) + beta C(r, :), or C_g = alpha
// sum_r A(r, :)^T B(r, :) + beta C_g, on v_mfma_f32_32x32x2_f32.
//
// Long groups are bound by the matrix cores (8 groups, 8192 rows by 2048 x 1024
// 130-132 TFLOP/s, the same rows as k of 1024 x 2048 134-136, the pipes 85-87%
// busy), short ones by reading B (16 groups, 24 rows by 2048 x 2048 5.2 TB/s),
// and what lies between partly by the rows that tiles pad to (64 groups of 64 rows
// on average by 1000 x 777 68 TFLOP/s, 81 with the padding).
//
// Edges.  An element outside op(A)'s rows or op(B)'s columns is fetched at an
// offset past the descriptor's end and reads as zero.  A partial last slice
// of k goes first, so that the main loop's loads need no test of k: an operand
// whose k runs along its stored rows ends at the last valid row, the other
// one compares each load's k (with 4-byte loads where K % 4 != 0, since a
// 16-byte one would hold values past K).  An operand with k down its columns
// and a width w that is no multiple of 4 has 16-byte loads whose last elements
// lie up to 3 past the width: they belong to rows or columns of the product
// that are not stored.  Such a load of row r reaches element 2 of row r + 1 at
// most (element 1 where w = 2), inside the operand for all rows but the last;
// so the last slice, partial or not, goes first with 4-byte loads.  (Width 1
// takes 4-byte loads throughout.)  63 groups, 3351 rows by 913 x 896: 110 us
// with 4-byte loads throughout, 102 so (tiles of 64 x 128, slices of 32).
#include "grouped.hpp"
#include "grouped_map.hpp"
#include "mfma_dma.hpp"

namespace sgemm {

namespace {

// Roundings of products of one sign add up along a chain of fused multiply-adds:
// u = 2^-24 of their sum for each.  So a chain has 128 k.  Up to 4096 k of a set
// of waves the chains are simply added: at most 128 + 31 u, and 3 for four sets,
// together 9.7e-6.  Beyond, what each addition rounds off goes into the next
// chain, whose 128 roundings see it: 134 u + K u^2, below 1e-5 up to K = 2^29.
// 8 groups, 8192 rows by 2048 x 1024: 260 us with one chain for a sum, 264 with
// chains added, 272 with the carry.
constexpr int kChain = 128, kPlain = 4096;

// KFORM: groups divide k (grouped_k; A^T and B as given); otherwise they
// divide the rows of A and C, and TB tells whether the B_g are stored
// transposed.  VA / VB: A / B take 16-byte loads.  KS sets of WM x WN waves
// share a tile; set q takes slices q, q + KS, .. through LDS stages of its own,
// and the sets' sums are added in order at the end.  STREAM: stores of C are
// non-temporal.
template <bool KFORM, bool TB, int BM, int BN, int BK, int WM, int WN, int KS, bool VA, bool VB,
          bool STREAM>
__global__ void __launch_bounds__(WM *WN *KS *kWave, 2)
grouped_kernel(GroupedArgs p, GroupMap map, FastDiv by_tiles, int tiles) {
  constexpr bool TA = KFORM;
  constexpr int NW = WM * WN;  // waves of a set
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  constexpr int KH = BK / 2, G = KH / 4;
  using GA = SliceGeom<BM, BK, TA, VA, true, NW>;
  using GB = SliceGeom<BN, BK, !TB, VB, true, NW>;
  static_assert(!GA::SPARE && !GB::SPARE, "loads must split evenly over the waves");
  constexpr int kLoads = GA::NBW + GB::NBW;

  constexpr int SA = BM * BK, SB = BK * BN;
  __shared__ __attribute__((aligned(1024))) float As0[KS * SA], As1[KS * SA];
  __shared__ __attribute__((aligned(1024))) float Bs0[KS * SB], Bs1[KS * SB];

  const int lane = threadIdx.x % kWave;
  const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int kq = KS > 1 ? all_waves / NW : 0;
  const int wave = KS > 1 ? all_waves % NW : all_waves;
  const int wm = wave / WN, wn = wave % WN;
  const int r32 = lane % 32, half = lane / 32;
  auto stage_a = [&](auto S) -> float * { return (decltype(S)::value ? As1 : As0) + kq * SA; };
  auto stage_b = [&](auto S) -> float * { return (decltype(S)::value ? Bs1 : Bs0) + kq * SB; };

  const float *A = p.A, *B = p.B;
  float *C = p.C;
  int m0, n0, m_end, K;
  if constexpr (KFORM) {
    // Each group's tiles are spread over the XCDs (a group of tiles per XCD
    // would leave the chip waiting for the XCD of the longest one), of up to 64
    // groups the longest first.
    const int rank = by_tiles((int)blockIdx.x);
    const int t = xcd_contiguous_id((int)blockIdx.x - rank * tiles, tiles);
    int first, last;
    const int g = group_by_length(p.offsets, p.groups, p.K, rank, first, last);
    A += first * p.lda;
    B += first * p.ldb;
    C += (long)g * p.strideC;
    K = last - first;
    const int tm = map.by_tiles_n(t);
    m0 = tm * BM;
    n0 = (t - tm * map.tiles_n) * BN;
    m_end = p.M;
  } else {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, BM, map);
    if (!t.valid) return;
    A += t.row0 * p.lda;
    B += (long)t.g * p.strideB;
    C += t.row0 * p.ldc;
    K = p.K;
    m0 = t.tm * BM;
    n0 = t.tn * BN;
    m_end = t.rows;
  }
  if (p.alpha == 0.f) K = 0;
  const float alpha = K > 0 ? p.alpha : 0.f;  // an empty sum is 0, whatever alpha is

  unsigned offA[GA::NBW], offB[GB::NBW];
#pragma unroll
  for (int q = 0; q < GA::NBW; ++q) {
    int row, col;
    GA::elem(wave, lane, q, row, col);
    offA[q] = m0 + GA::mnof(row, col) < m_end ? (unsigned)(row * p.lda + col) * 4u : kOutOfRange;
  }
#pragma unroll
  for (int q = 0; q < GB::NBW; ++q) {
    int row, col;
    GB::elem(wave, lane, q, row, col);
    offB[q] = n0 + GB::mnof(row, col) < p.N ? (unsigned)(row * p.ldb + col) * 4u : kOutOfRange;
  }
  auto rsrc = [](const float *base, int records) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(base), 0, records,
                                             kRawBufferWord3);
  };
  auto origin_a = [&](int k0) { return TA ? A + (long)k0 * p.lda + m0 : A + (long)m0 * p.lda + k0; };
  auto origin_b = [&](int k0) { return TB ? B + (long)n0 * p.ldb + k0 : B + (long)k0 * p.ldb + n0; };

  // Position u of the slice order: with a ragged K or edge the last slice first,
  // then slice u - 1.  Positions at or past nk get descriptors without
  // records: nothing is fetched.
  const bool wide_edge = (TA && VA && p.M % 4 != 0) || (!TB && VB && p.N % 4 != 0);
  const int nk = (K + BK - 1) / BK, ragged = K % BK != 0 || wide_edge;
  auto dma = [&](auto S, int u) {
    const int records = u < nk ? kBufferRecords : 0;
    const int k0 = u < nk ? (u - ragged) * BK : 0;
    const __amdgpu_buffer_rsrc_t ra = rsrc(origin_a(k0), records);
    const __amdgpu_buffer_rsrc_t rb = rsrc(origin_b(k0), records);
#pragma unroll
    for (int q = 0; q < GA::NBW; ++q)
      lds_dma<VA>(ra, stage_a(S) + (wave + q * NW) * GA::FPB, offA[q]);
#pragma unroll
    for (int q = 0; q < GB::NBW; ++q)
      lds_dma<VB>(rb, stage_b(S) + (wave + q * NW) * GB::FPB, offB[q]);
  };
  // The last slice, kl values of k, into stage 0.
  auto dma_tail = [&](auto geom, float *stage, const float *origin, long ld, int mn_left, int kl) {
    using Gm = decltype(geom);
    const __amdgpu_buffer_rsrc_t r = rsrc(origin, Gm::KR ? kl * (int)ld * 4 : kBufferRecords);
#pragma unroll
    for (int q = 0; q < Gm::NBW; ++q) {
      int row, col;
      Gm::elem(wave, lane, q, row, col);
      const bool in = Gm::mnof(row, col) < mn_left && (Gm::KR || Gm::kof(row, col) < kl);
      lds_dma<Gm::E == 4>(r, stage + (wave + q * NW) * Gm::FPB,
                          in ? (unsigned)(row * ld + col) * 4u : kOutOfRange);
    }
  };

  const int sw = kc_swizzle<BK, true>(r32);
  int a_off[G], b_off[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    a_off[g] = TA ? (half * KH + g * 4) * BM + wm * WTM + r32
                  : (wm * WTM + r32) * BK + 4 * ((half * (KH / 4) + g) ^ sw);
    b_off[g] = TB ? (wn * WTN + r32) * BK + 4 * ((half * (KH / 4) + g) ^ sw)
                  : (half * KH + g * 4) * BN + wn * WTN + r32;
  }
  struct Ops {
    f32x4 a[FM], b[FN];
  };
  auto read_ops = [&](auto S, int g, Ops &o) {
    const float *as = stage_a(S), *bs = stage_b(S);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (TA) {
#pragma unroll
        for (int t = 0; t < 4; ++t) o.a[i][t] = as[a_off[g] + t * BM + i * 32];
      } else {
        o.a[i] = *reinterpret_cast<const f32x4 *>(as + a_off[g] + i * 32 * BK);
      }
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (TB) {
        o.b[j] = *reinterpret_cast<const f32x4 *>(bs + b_off[g] + j * 32 * BK);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) o.b[j][t] = bs[b_off[g] + t * BN + j * 32];
      }
    }
  };
  f32x16 acc[FM][FN], sum[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = sum[i][j][e] = 0.f;
  auto mma = [&](const Ops &o) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma32x32x2(o.a[i][t], o.b[j][t], acc[i][j]);
  };
  // A chain ends in `sum`; the next one begins with 0, or, with CARRY, with what
  // the addition rounded off (once it is not finite, 0: an infinity stays one).
  auto end_chain = [&](auto CARRY) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float before = sum[i][j][e];
          sum[i][j][e] += acc[i][j][e];
          if constexpr (decltype(CARRY)::value)
            acc[i][j][e] = __builtin_isfinite(sum[i][j][e])
                               ? acc[i][j][e] - (sum[i][j][e] - before) : 0.f;
          else
            acc[i][j][e] = 0.f;
        }
  };

  // As in mfma_dma.hpp: one matrix-core instruction per load in the last group
  // of a slice, then two per operand read.
  constexpr int kMfma = 4 * FM * FN;
  constexpr int kReads = (TA ? 2 * FM : FM) + (TB ? FN : 2 * FN);
  auto interleave = [&](auto last) {
    constexpr int loads = decltype(last)::value ? kLoads : 0;
    static_for<kMfma>([&](auto I) {
      constexpr int i = decltype(I)::value;
      constexpr int d = kReads * (i + 1) / kMfma - kReads * i / kMfma;
      constexpr int v = loads * (i + 1) / kMfma - loads * i / kMfma;
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
      if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);
    });
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  Ops cur, nxt;
  auto slice = [&](auto S, int t) {  // the set's t-th slice
    using SN = std::integral_constant<int, 1 - decltype(S)::value>;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g + 1 < G) {
        read_ops(S, g + 1, nxt);
        mma(cur);
        interleave(std::false_type());
      } else {
        dma_barrier_keep<0>();
        dma(S, kq + (t + 2) * KS);
        read_ops(SN(), 0, nxt);
        mma(cur);
        interleave(std::true_type());
      }
      cur = nxt;
    }
  };

  if (nk > 0) {
    const int turns = (nk + KS - 1) / KS;  // the same for all sets: they share the barriers
    if (ragged && kq == 0) {
      const int k0 = (nk - 1) * BK, kl = K - k0;
      using GAn = SliceGeom<BM, BK, TA, false, true, NW>;
      using GBn = SliceGeom<BN, BK, !TB, false, true, NW>;
      if (TA ? p.M % 4 != 0 : K % 4 != 0)
        dma_tail(GAn(), stage_a(S0()), origin_a(k0), p.lda, m_end - m0, kl);
      else
        dma_tail(GA(), stage_a(S0()), origin_a(k0), p.lda, m_end - m0, kl);
      if (TB ? K % 4 != 0 : p.N % 4 != 0)
        dma_tail(GBn(), stage_b(S0()), origin_b(k0), p.ldb, p.N - n0, kl);
      else
        dma_tail(GB(), stage_b(S0()), origin_b(k0), p.ldb, p.N - n0, kl);
    } else {
      dma(S0(), kq);
    }
    dma(S1(), kq + KS);
    dma_barrier_keep<kLoads>();
    read_ops(S0(), 0, cur);
    constexpr int kTurns = kChain / BK;  // of a chain
    static_assert(kTurns % 2 == 0, "a chain begins with stage 0");
    auto chains = [&](auto CARRY) __attribute__((always_inline)) {
      for (int t = 0; t < turns;) {
        const int end = min(t + kTurns, turns);
        for (; t < end; t += 2) {
          slice(S0(), t);
          if (t + 1 < end) slice(S1(), t + 1);
        }
        end_chain(CARRY);
      }
    };
    if (turns <= kPlain / BK) {
      chains(std::false_type());
    } else {
      chains(std::true_type());
      end_chain(std::false_type());
    }
    // The last slices sent loads past K (no memory traffic): let them retire
    // before the work-group gives up its LDS.
    __builtin_amdgcn_s_waitcnt(0x0f70);
  }

  if constexpr (KS > 1) {
    // The stages are free: every load has landed, every operand has been read.
    // Set s > 0 leaves its sums in As0, those that do not fit there in Bs0.
    constexpr int kSums = NW * FM * FN * 16 * kWave, kInA = KS * SA / kSums;
    static_assert(kInA + KS * SB / kSums >= KS - 1, "the sets' sums fit the first stages");
    __syncthreads();
    auto sums = [&](int set, int i, int j) {
      float *const at = set - 1 < kInA ? As0 + (set - 1) * kSums : Bs0 + (set - 1 - kInA) * kSums;
      return at + ((wave * FM + i) * FN + j) * 16 * kWave + lane;
    };
    if (kq > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) sums(kq, i, j)[e * kWave] = sum[i][j][e];
    }
    __syncthreads();
    if (kq > 0) return;
#pragma unroll
    for (int set = 1; set < KS; ++set)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[i][j][e] += sums(set, i, j)[e * kWave];
  }

  // Register e of lane l holds row acc32_row(l, e), column l % 32 of a block:
  // row 4 (l / 32) of a uniform base and a constant number of rows past it.
  const bool full = m0 + BM <= m_end && n0 + BN <= p.N;
  const int mw = m0 + wm * WTM, nw = n0 + wn * WTN;
  float *const origin = C + (long)mw * p.ldc + nw;
  const unsigned lane_at = (unsigned)(4 * half * p.ldc + r32) * 4u;
  const int rows = m_end - mw - 4 * half, cols = p.N - nw - r32;
  auto store = [&](auto whole, auto with_c) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = i * 32 + 8 * (e >> 2) + (e & 3);
        float *const row = origin + r * p.ldc;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (!decltype(whole)::value && (r >= rows || j * 32 >= cols)) continue;
          float *const at =
              reinterpret_cast<float *>(reinterpret_cast<char *>(row + j * 32) + lane_at);
          const float v = sum[i][j][e];
          if constexpr (decltype(with_c)::value)
            *at = fmaf(alpha, v, p.beta * *at);
          else if constexpr (STREAM)
            __builtin_nontemporal_store(alpha * v, at);
          else
            *at = alpha * v;
        }
      }
  };
  if (p.beta != 0.f)
    store(std::false_type(), std::true_type());
  else if (full)
    store(std::true_type(), std::false_type());
  else
    store(std::false_type(), std::false_type());
}

template <bool KFORM, bool TB, int BM, int BN, int BK, int WM, int WN, int KS, bool VA, bool VB,
          bool STREAM = true>
hipError_t launch(const GroupedArgs &p, hipStream_t s) {
  const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  const long rows = KFORM ? (long)tiles_m * p.groups : group_tile_rows(p.M, p.groups, BM);
  hipLaunchKernelGGL((grouped_kernel<KFORM, TB, BM, BN, BK, WM, WN, KS, VA, VB, STREAM>),
                     dim3((unsigned)(rows * tiles_n)), dim3(WM * WN * KS * kWave), 0, s, p,
                     make_group_map(tiles_n), make_fast_div(tiles_m * tiles_n), tiles_m * tiles_n);
  return hipGetLastError();
}

template <int BM, int BN, int BK, int WM, int WN, int KS>
hipError_t launch_rows(const GroupedArgs &p, bool tb, hipStream_t s) {
  if (tb) return launch<false, true, BM, BN, BK, WM, WN, KS, true, true>(p, s);
  if (p.N > 1) return launch<false, false, BM, BN, BK, WM, WN, KS, true, true>(p, s);
  return launch<false, false, 32, 32, 32, 1, 1, 4, true, false>(p, s);
}

template <int BM, int BN, int BK, int WM, int WN, int KS, bool STREAM = true>
hipError_t launch_k(const GroupedArgs &p, hipStream_t s) {
  if (p.M > 1 && p.N > 1)
    return launch<true, false, BM, BN, BK, WM, WN, KS, true, true, STREAM>(p, s);
  return launch<true, false, 32, 32, 32, 1, 1, 4, false, false>(p, s);
}

}  // namespace

// Four tiles; `small` is the number of 32 x 32 ones, as far as the host knows
// it (to within the groups' lengths).
//  - 32 x 32, 4 sets of waves over k in slices of 32: where few work-groups
//    each have a long sum, latency bounds them, and more waves on a sum hide it.
//  - the same in slices of 16 for groups of a few rows, some of them empty:
//    reading B bounds them, and 32 KiB of LDS for 64 let twice as many
//    work-groups read.
//  - 32 x 64, 2 sets: groups that would leave much of a 64-row tile empty, and
//    products whose 64 x 64 tiles would be few.
//  - 64 x 64: the least LDS traffic per product of the four.
// Measured in that order (us; B as given and not in the caches, groups of
// unequal length):
//    1 group of 1 row by 8192 x 8192       67   89  110  191
//    1 of 64 by 4096 x 4096                35   46   55   97
//    16 groups, 24 rows by 2048 x 2048     49   37   43   74
//    32 groups, 24 rows by 1024 x 2048     44   34   42   74
//    64 groups, 512 rows by 1024 x 1024    59   53   60   68
//    16 groups, 128 rows by 2048 x 2048    53   53   45   75
//    16 groups, 512 rows by 2048 x 2048    79   84   63  101
//    4 groups, 200 rows by 2000 x 4000     52   53   60  100
//    the same, other lengths               74   60   76   99
//    8 groups, 2048 rows by 2048 x 1024   107   90   84   92
//    8 groups, 8192 rows by 2048 x 1024   363  308  284  268
hipError_t launch_grouped_rows(const GroupedArgs &p, bool tb, int cus, hipStream_t s) {
  const long groups = p.groups < p.M ? p.groups : p.M, most = p.M / 32 + groups / 2;
  const long small = (most > groups ? most : groups) * ((p.N + 31) / 32);
  const long mean = p.M / p.groups;
  if (small <= cus || (mean >= 8 && 2 * small <= 5L * cus))
    return launch_rows<32, 32, 32, 1, 1, 4>(p, tb, s);
  if (mean < 8 || (mean < 16 && small > 6L * cus)) return launch_rows<32, 32, 16, 1, 1, 4>(p, tb, s);
  if (mean < 192 || small < 12L * cus) return launch_rows<32, 64, 32, 1, 2, 2>(p, tb, s);
  return launch_rows<64, 64, 32, 2, 2, 1>(p, tb, s);
}

// Tiles of 64 x 128 in slices of 16 rows (24 KiB of LDS and 120 registers: four
// work-groups of a compute unit hide each other's start and end, and groups are
// padded less)
// where there are 4 for every compute unit; else 64 x 64, but 32 x 32 with 4
// sets of waves over the rows where those leave compute units without a tile
// and the groups are long.  Measured in that order (us):
//    8 groups, 8192 rows by 1024 x 2048         261   278   423
//    63 groups, 3351 rows by 913 x 896           82   111   411
//    32 groups, 1500 rows by 257 x 1000          19    23    78
//    12 groups, 4096 rows by 512 x 1024          51    43    83
//    8 groups, 1024 rows by 256 x 512            16    10    12
//    3 groups, 4096 rows by 512 x 512           107    56    30
//    1 group of 16384 rows by 64 x 64           760   392   124
hipError_t launch_grouped_k(const GroupedArgs &p, int cus, hipStream_t s) {
  const long m64 = (p.M + 63) / 64, n128 = (p.N + 127) / 128, n64 = (p.N + 63) / 64;
  // Groups of a few rows leave little but the writing of C.  Unless each row of C
  // starts on 64 bytes, stores are then better not streamed: parts of a line
  // meet in L2.  Streamed / plain at 2, 16, 24, 33 and 64 rows a group:
  //    24 groups, 512 x 1544   27/21  28/25  29/28  30/31  38/40
  //    49 groups, 192 x 2667   48/32  48/36  49/37  48/41  55/52
  //    49 groups, 192 x 2688   21/23  23/29  25/31  29/37  40/48
  //    the same, C 32 bytes on 46/30  47/34  48/37  49/41  55/51
  //    32 groups, 257 x 1000   13/13  16/17  17/18  17/20  20/25
  const bool lines =
      ((reinterpret_cast<uintptr_t>(p.C) / 4 | p.ldc | (p.groups > 1 ? p.strideC : 0)) & 15) == 0;
  const bool stream = lines || p.K > 32L * p.groups;
  if (m64 * n128 * p.groups >= 4L * cus)
    return stream ? launch_k<64, 128, 16, 2, 2, 1>(p, s)
                  : launch_k<64, 128, 16, 2, 2, 1, false>(p, s);
  if (2 * m64 * n64 * p.groups > 3L * cus || p.K < 192L * p.groups)
    return launch_k<64, 64, 32, 2, 2, 1>(p, s);
  return launch_k<32, 32, 32, 1, 1, 4>(p, s);
}

}  // namespace sgemm
