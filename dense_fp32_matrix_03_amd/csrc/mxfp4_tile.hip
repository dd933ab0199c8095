// mxfp4_tile.hip -- products of matrices held in microscaled 4-bit floating
// point whose operand slices reach LDS by buffer-to-LDS loads.
//
// C(m, n) = alpha sum_b 2^(sa(m, b) + sb(n, b) - 254) sum_{k in b} a(m, k) b(n, k)
// + beta C(m, n), on v_mfma_scale_f32_32x32x64_f8f6f4: 32 rows of A by 32 rows
// of B over 64 k, lane half h supplying one block of 32 codes (16 bytes) of row
// l % 32 of each operand and its scale byte, which op_sel picks from the four
// bytes of a register.
//
// A slice is 256 k, two granules: 128 bytes of codes and two dwords of scales a
// row.  Half h has granule h of the slice and instruction s its block s, so one
// dword of scales serves a lane for the slice's four instructions.  The codes'
// LDS image is [row][8 chunks of 16 bytes], chunk c at c ^ kc_swizzle
// (mfma_dma.hpp), the scales' [granule][row].
//
// 8192^3 with bfloat16 C takes 260-290 us, 3.8-4.2 PFLOP/s at an engine clock of
// 1.85-2.1 GHz.  The main loop runs at 5 PFLOP/s, what the 4-bit instructions
// alone sustain on such data (5.0-5.8, at 1.5 GHz: power decides); the rest
// is the burst of C's stores, in which the matrix cores idle.  Smaller products
// are bound by the first loads and the stores of a tile, and short groups by
// reading B (32 groups, 48 rows by 4096 x 2048 4.1 TB/s).
//
// Accuracy.  An instruction drops the products below 2^-27 of its largest addend
// (measured: 64 products of 1.5 2^-28 added to 1 leave 1, those of 1.5 2^-27 are
// all there) and rounds once, so that a sum is off by at most (9 K / 64 + 12)
// 2^-24 of sum |products|.  A second level of sums would take away the roundings,
// an eighth of that, and the 256 x 256 tile's last registers; the drops need one
// every ten instructions.  Codes of neighbouring scales sum exactly: nothing is
// lost on normally distributed operands up to K = 32768.
//
// Edges.  The descriptors end at the last row's last byte, so rows past it
// read as zeros.  Where K ends inside a slice the second granule's codes are
// whatever follows in memory, below that end (every code is finite), but both
// operands' scales there read as 0: the products are at most 36 2^-254 and
// vanish in single precision.
#include <math.h>

#include "grouped_map.hpp"
#include "mfma_dma.hpp"
#include "mxfp4.hpp"

namespace sgemm {

namespace {

constexpr int kSliceBytes = 128;  // codes of a row's slice

// KS sets of WM x WN waves share a tile; set q takes slices q, q + KS, ..
// through LDS stages of its own, and the sets' sums are added in order at the
// end.  With few tiles the time is a chain of slices, each as long as its
// loads take to arrive: the sets walk KS chains at once.
template <int BM, int BN, int WM, int WN, int KS, bool CBF16>
__global__ void __launch_bounds__(WM *WN *KS *kWave, 2)
mxfp4_tile_kernel(Mxfp4Args p, TileMap tmap, GroupMap map) {
  constexpr int NW = WM * WN;  // waves of a set
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  constexpr int QA = BM * kSliceBytes / 1024 / NW, QB = BN * kSliceBytes / 1024 / NW;
  // Loads of 64 rows' scales of a granule.  Where they do not split evenly, some waves'
  // last one is spare: it reads nothing, into LDS that nobody reads, so that
  // every wave has the same number of loads in flight.
  constexpr int US = (BM + BN) / 32, QS = (US + NW - 1) / NW;
  static_assert(QA * NW * 1024 == BM * kSliceBytes && QB * NW * 1024 == BN * kSliceBytes,
                "loads must split evenly over the waves");
  constexpr int kLoads = QA + QB + QS;

  // One LDS array per stage and operand, so that the compiler sees that loads
  // into one stage do not touch the one that is read (mfma_dma.hpp).
  constexpr int SA = BM * kSliceBytes / 4, SB = BN * kSliceBytes / 4, SS = QS * NW * 64;
  __shared__ __attribute__((aligned(1024))) float As0[KS * SA], As1[KS * SA];
  __shared__ __attribute__((aligned(1024))) float Bs0[KS * SB], Bs1[KS * SB];
  // Scales: A's rows, then B's.
  __shared__ __attribute__((aligned(1024))) float Ss0[KS * SS], Ss1[KS * SS];

  const int lane = threadIdx.x % kWave;
  const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int kq = KS > 1 ? all_waves / NW : 0;
  const int wave = KS > 1 ? all_waves % NW : all_waves;
  const int wm = wave / WN, wn = wave % WN;
  const int r32 = lane % 32, half = lane / 32;
  auto stage_a = [&](auto S) -> float * { return (decltype(S)::value ? As1 : As0) + kq * SA; };
  auto stage_b = [&](auto S) -> float * { return (decltype(S)::value ? Bs1 : Bs0) + kq * SB; };
  auto stage_s = [&](auto S) -> float * { return (decltype(S)::value ? Ss1 : Ss0) + kq * SS; };

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
  const int granules = (p.K + 127) / 128;
  const int pitch = granules * 64;  // bytes of a row's codes
  const int rows_a = min(BM, m_end - m0), rows_b = min(BN, p.N - n0);
  const unsigned char *a0 = p.a.codes + (a_row + m0) * pitch;
  const unsigned char *b0 = p.b.codes + (b_row + n0) * pitch;
  const unsigned *sa0 = p.a.scales + a_row + m0;
  const unsigned *sb0 = p.b.scales + b_row + n0;

  // Load q of a wave fetches rows 8 (wave + q NW) .. + 7 of the slice, of
  // either operand: one set of lane offsets serves both.
  constexpr int Q = QA > QB ? QA : QB;
  unsigned off[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int row = 8 * (wave + q * NW) + lane / 8;
    off[q] = (unsigned)(row * pitch + 16 * ((lane % 8) ^ kc_swizzle<32, true>(row)));
  }

  const int nk = (granules + 1) / 2;
  auto rsrc = [](const void *base, int records) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, records,
                                             kRawBufferWord3);
  };
  // Loads of the set's next slice into stage S.  Slices at or past nk get
  // descriptors without records: nothing is fetched.  No branch depends on
  // that, so that the loads can be scheduled between matrix-core instructions.
  int k = kq;  // the slice
  const unsigned *s_base[QS];
  long s_lds[QS];
  unsigned s_off[QS];
  int s_records[QS], s_granule[QS];
#pragma unroll
  for (int q = 0; q < QS; ++q) {
    const int u = wave + q * NW;  // uniform: which 64 rows of which granule
    const bool of_a = u < BM / 32;
    const int v = of_a ? u : u - BM / 32, per = of_a ? BM / 64 : BN / 64;
    s_lds[q] = of_a ? p.a.lds : p.b.lds;
    s_granule[q] = v / per;
    s_base[q] = of_a ? sa0 : sb0;
    s_off[q] = (unsigned)(v % per * 64 + lane) * 4u;
    s_records[q] = u < US ? 4 * (of_a ? rows_a : rows_b) : 0;
  }
  auto dma = [&](auto S) {
    const bool live = k < nk;
    const int k0 = k * kSliceBytes;
    const __amdgpu_buffer_rsrc_t ra = rsrc(a0 + k0, live ? rows_a * pitch - k0 : 0);
    const __amdgpu_buffer_rsrc_t rb = rsrc(b0 + k0, live ? rows_b * pitch - k0 : 0);
#pragma unroll
    for (int q = 0; q < QA; ++q) lds_dma<true>(ra, stage_a(S) + (wave + q * NW) * 256, off[q]);
#pragma unroll
    for (int q = 0; q < QB; ++q) lds_dma<true>(rb, stage_b(S) + (wave + q * NW) * 256, off[q]);
#pragma unroll
    for (int q = 0; q < QS; ++q) {
      const int g = 2 * k + s_granule[q];
      lds_dma<false>(rsrc(s_base[q] + g * s_lds[q], g < granules ? s_records[q] : 0),
                     stage_s(S) + (wave + q * NW) * 64, s_off[q]);
    }
    k += KS;
  };

  const int sw = kc_swizzle<32, true>(r32);
  struct Ops {
    i32x4 a[FM], b[FN];
  };
  struct Scales {
    int a[FM], b[FN];
  };
  auto read_ops = [&](auto S, int s, Ops &o) {
    const int ch = ((4 * half + s) ^ sw) * 4;
#pragma unroll
    for (int i = 0; i < FM; ++i)
      o.a[i] = *reinterpret_cast<const i32x4 *>(stage_a(S) + (wm * WTM + i * 32 + r32) * 32 + ch);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      o.b[j] = *reinterpret_cast<const i32x4 *>(stage_b(S) + (wn * WTN + j * 32 + r32) * 32 + ch);
  };
  auto read_scales = [&](auto S, Scales &c) {
    const int *sa = reinterpret_cast<const int *>(stage_s(S)) + half * BM + wm * WTM + r32;
    const int *sb = reinterpret_cast<const int *>(stage_s(S)) + 2 * BM + half * BN + wn * WTN + r32;
#pragma unroll
    for (int i = 0; i < FM; ++i) c.a[i] = sa[i * 32];
#pragma unroll
    for (int j = 0; j < FN; ++j) c.b[j] = sb[j * 32];
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  Scales sc, sn;
  auto mma = [&](auto STEP, const Ops &o) {
    constexpr int s = decltype(STEP)::value;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = mfma_fp4_32x32x64<s>(o.a[i], o.b[j], acc[i][j], sc.a[i], sc.b[j]);
  };

  // A step's operand reads (and a slice's loads) are spread between its
  // matrix-core instructions.
  constexpr int kMfma = FM * FN, kReads = FM + FN;
  auto interleave = [&](auto last) {
    constexpr int loads = decltype(last)::value ? kLoads : 0;
    constexpr int reads = kReads + (decltype(last)::value ? (FM + 1) / 2 + (FN + 1) / 2 : 0);
    static_for<kMfma>([&](auto I) {
      constexpr int i = decltype(I)::value;
      constexpr int v = loads * (i + 1) / kMfma - loads * i / kMfma;
      constexpr int d = reads * (i + 1) / kMfma - reads * i / kMfma;
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // matrix core
      if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);  // DS read
      if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);  // VMEM read
    });
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  // The set's t-th slice is in stage S, the next one on its way to the
  // other.
  // WHOLE: a wave with one block of 32 x 32 has too few matrix-core
  // instructions in a step to cover the next one's reads, and registers to
  // spare: it reads a whole slice's operands while it multiplies the one
  // before.  The barrier waits for slice t + 1, and for every wave to have read
  // slice t; then slice t + 2 goes to stage S.
  // Otherwise the operands are read a step ahead, and the last step of a slice
  // waits for slice t + 1, and for every wave to be done with stage S, sends
  // slice t + 2 there and reads slice t + 1's first operands.
  constexpr bool WHOLE = FM * FN == 1;
  constexpr int kAhead = WHOLE ? 4 : 1;  // steps whose operands are held
  Ops cur[kAhead], nxt[kAhead];
  auto read_ahead = [&](auto S, Ops *o) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) read_ops(S, s, o[s]);
  };
  auto slice = [&](auto S) {
    using SN = std::integral_constant<int, 1 - decltype(S)::value>;
    if constexpr (WHOLE) {
      dma_barrier_keep<0>();
      dma(S);
      read_ahead(SN(), nxt);
      read_scales(SN(), sn);
      static_for<4>([&](auto STEP) { mma(STEP, cur[decltype(STEP)::value]); });
#pragma unroll
      for (int s = 0; s < kAhead; ++s) cur[s] = nxt[s];
    } else {
      static_for<4>([&](auto STEP) {
        constexpr int s = decltype(STEP)::value;
        if constexpr (s < 3) {
          read_ops(S, s + 1, nxt[0]);
          mma(STEP, cur[0]);
          interleave(std::false_type());
        } else {
          dma_barrier_keep<0>();
          dma(S);
          read_ops(SN(), 0, nxt[0]);
          read_scales(SN(), sn);
          mma(STEP, cur[0]);
          interleave(std::true_type());
        }
        cur[0] = nxt[0];
      });
    }
    sc = sn;
  };

  if (nk > 0) {
    const int turns = (nk + KS - 1) / KS;  // the same for all sets: they share the barriers
    dma(S0());
    dma(S1());
    dma_barrier_keep<kLoads>();
    read_ahead(S0(), cur);
    read_scales(S0(), sc);
    for (int t = 0; t < turns; t += 2) {
      slice(S0());
      if (t + 1 < turns) slice(S1());
    }
    // The last slices sent loads past K (no memory traffic): let them retire
    // before the work-group gives up its LDS.
    __builtin_amdgcn_s_waitcnt(0x0f70);
  }

  if constexpr (KS > 1) {
    // The stages are free: every load has landed, every operand has been read.
    // Set s > 0 leaves its sums at 4 KiFloat (s - 1) of As0, the last of four
    // sets in Bs0.
    static_assert(FM * FN * NW == 4 && (KS == 2 || KS == 4) && KS * SA == 2048 * KS &&
                      SB == SA, "a set's sums are 16 KiB");
    __syncthreads();
    auto sums = [&](int set) { return (set == 3 ? Bs0 : As0 + (set - 1) * 4096) + wave * 1024 + lane; };
    if (kq > 0) {
      float *at = sums(kq);
#pragma unroll
      for (int e = 0; e < 16; ++e) at[e * kWave] = acc[0][0][e];
    }
    __syncthreads();
    if (kq > 0) return;
#pragma unroll
    for (int set = 1; set < KS; ++set)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[0][0][e] += sums(set)[e * kWave];
  }

  // Register e of lane l holds row acc32_row(l, e), column l % 32 of a block:
  // row 4 (l / 32) of a uniform base and a constant number of rows past it.
  // Stores of the smaller tiles are non-temporal (2048^3 10.3 -> 9.4 us on 128 x
  // 128 tiles with bfloat16 C, 11.1 -> 9.6 on 64 x 64 with FP32); the 256 x 256
  // tile's, bursts of a whole chip's tiles at once, are not (8192^2 x 1024 55
  // against 75 us, 8192^3 259 against 270).  Passing the rows through LDS for
  // stores of 16 bytes a lane took 1.5 us more a tile.
  using T = std::conditional_t<CBF16, __bf16, float>;
  const bool full = m0 + BM <= m_end && n0 + BN <= p.N;
  const int mw = m0 + wm * WTM, nw = n0 + wn * WTN;
  T *const origin = static_cast<T *>(p.C) + (a_row + mw) * p.ldc + nw;
  const unsigned lane_at = (unsigned)((4 * half * p.ldc + r32) * sizeof(T));
  const int rows = m_end - mw - 4 * half, cols = p.N - nw - r32;
  auto store = [&](auto whole, auto with_c) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = i * 32 + 8 * (e >> 2) + (e & 3);
        T *const row = origin + r * p.ldc;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (!decltype(whole)::value && (r >= rows || j * 32 >= cols)) continue;
          T *const at = reinterpret_cast<T *>(reinterpret_cast<char *>(row + j * 32) + lane_at);
          const float v = acc[i][j][e];
          if constexpr (decltype(with_c)::value)
            *at = (T)fmaf(p.alpha, v, p.beta * (float)*at);
          else if constexpr (BM < 256)
            __builtin_nontemporal_store((T)(p.alpha * v), at);
          else
            *at = (T)(p.alpha * v);
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

template <int BM, int BN, int WM, int WN, int KS>
hipError_t launch(const Mxfp4Args &p, bool c_bf16, hipStream_t s) {
  const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  const long rows = p.offsets ? group_tile_rows(p.M, p.groups, BM) : tiles_m;
  const dim3 grid((unsigned)(rows * tiles_n)), block(WM * WN * KS * kWave);
  const TileMap tmap = make_tile_map(tiles_m, tiles_n, kGroupRaster);
  const GroupMap map = make_group_map(tiles_n);
  if (c_bf16)
    hipLaunchKernelGGL((mxfp4_tile_kernel<BM, BN, WM, WN, KS, true>), grid, block, 0, s, p, tmap,
                       map);
  else
    hipLaunchKernelGGL((mxfp4_tile_kernel<BM, BN, WM, WN, KS, false>), grid, block, 0, s, p, tmap,
                       map);
  return hipGetLastError();
}

}  // namespace

// Groups count with their mean length: the host does not know more.  In units
// of a round of 256 x 256 tiles (one on each compute unit), a compute unit
// takes for n tiles
//   of 128 x 128   0.65 (n = 1), 0.77 (2), 0.29 n (more: two share the unit),
//   of 64 x 64     0.35 (1), 0.42 (2), 0.16 n (more).
// Measured on 256 compute units with bfloat16 C and K = 8192 (N = 8192), 64 x
// 64 / 128 x 128 / 256 x 256: M = 128 25 / 39 / 64 us, 256 27 / 39 / 65, 512
// 42 / 39 / 64, 1024 74 / 47 / 64, 8192 464 / 346 / 289; 2048 x 4096 x 4096
// 39 / 24 / 33; 16 groups, 8192 rows by 2048 x 2048 53 / 43 / 46.  Groups of up
// to 64 rows are bound by reading B, which the smallest tile does best: 32
// groups, 48 rows by 4096 x 2048 27 / 31 / 42.  Sets of waves on the 64 x 64
// tile, 1 / 2 / 4 of them: 128 x 8192 x 8192 17.5 / 14.7 / 13.2 us, 64 x 4096 x
// 14336 21.7 / 17.9 / 15.6, 117 x 1785 x 5632 8.5 / 8.4 / 9.1; 256 x 8192 x 8192
// 27 / 24, with four one work-group fills a compute unit.
hipError_t launch_mxfp4_tile(const Mxfp4Args &p, bool c_bf16, int cus, hipStream_t s) {
  const long groups = !p.offsets ? 1 : p.groups < p.M ? p.groups : p.M;
  const double mean = (double)p.M / groups;
  auto per_cu = [&](long t) {
    const double rows = p.offsets ? fmax(1.0, mean / t + 0.5) : ceil(mean / t);
    return ceil(groups * rows * ((p.N + t - 1) / t) / cus);
  };
  const double n64 = per_cu(64), n128 = per_cu(128);
  const double c64 = n64 == 1 ? 0.35 : n64 == 2 ? 0.42 : 0.16 * n64;
  const double c128 = n128 == 1 ? 0.65 : n128 == 2 ? 0.77 : 0.29 * n128;
  if ((p.offsets && mean <= 64) || (c64 <= c128 && c64 <= per_cu(256))) {
    if (n64 == 1 && p.K >= 6144) return launch<64, 64, 2, 2, 4>(p, c_bf16, s);
    if (n64 == 2 && p.K >= 6144) return launch<64, 64, 2, 2, 2>(p, c_bf16, s);
    return launch<64, 64, 2, 2, 1>(p, c_bf16, s);
  }
  return c128 <= per_cu(256) ? launch<128, 128, 2, 2, 1>(p, c_bf16, s)
                             : launch<256, 256, 2, 4, 1>(p, c_bf16, s);
}

}  // namespace sgemm
