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
// Edges.  The descriptors end at the last row's last byte, so rows past it
// read as zeros.  Where K ends inside a slice the second granule's codes are
// whatever follows in memory, below that end (every code is finite), but both
// operands' scales there read as 0: the products are at most 36 2^-254 and
// vanish in single precision.
#include "grouped_map.hpp"
#include "mfma_dma.hpp"
#include "mxfp4.hpp"

namespace sgemm {

namespace {

constexpr int kSliceBytes = 128;  // codes of a row's slice

template <int BM, int BN, int WM, int WN, int NST, bool CBF16>
__global__ void __launch_bounds__(WM *WN *kWave, 2)
mxfp4_tile_kernel(Mxfp4Args p, TileMap tmap, int tiles_n) {
  constexpr int NW = WM * WN;
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
  static_assert(NST >= 2 && NST <= 4, "2 to 4 LDS stages");
  constexpr int SA = BM * kSliceBytes / 4, SB = BN * kSliceBytes / 4, SS = QS * NW * 64;
  __shared__ __attribute__((aligned(1024))) float As0[SA], As1[SA], As2[NST > 2 ? SA : 1],
      As3[NST > 3 ? SA : 1];
  __shared__ __attribute__((aligned(1024))) float Bs0[SB], Bs1[SB], Bs2[NST > 2 ? SB : 1],
      Bs3[NST > 3 ? SB : 1];
  __shared__ __attribute__((aligned(1024))) float Ss0[SS], Ss1[SS], Ss2[NST > 2 ? SS : 1],
      Ss3[NST > 3 ? SS : 1];  // scales: A's rows, then B's
  auto stage_a = [&](auto S) -> float * {
    constexpr int i = decltype(S)::value;
    return i == 0 ? As0 : i == 1 ? As1 : i == 2 ? As2 : As3;
  };
  auto stage_b = [&](auto S) -> float * {
    constexpr int i = decltype(S)::value;
    return i == 0 ? Bs0 : i == 1 ? Bs1 : i == 2 ? Bs2 : Bs3;
  };
  auto stage_s = [&](auto S) -> float * {
    constexpr int i = decltype(S)::value;
    return i == 0 ? Ss0 : i == 1 ? Ss1 : i == 2 ? Ss2 : Ss3;
  };

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int r32 = lane % 32, half = lane / 32;

  long a_row = 0, b_row = 0;  // first row of the group in A (and C), and of its B
  int m0, n0, m_end = p.M;
  if (p.offsets) {
    const GroupTile t = group_tile(p.offsets, p.groups, p.M, BM, tiles_n, 8);
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
  // Slices at or past nk get descriptors without records: nothing is fetched.
  // No branch depends on that, so that the loads can be scheduled between
  // matrix-core instructions.
  auto dma = [&](auto S, int t) {
    const bool live = t < nk;
    const long k0 = (long)t * kSliceBytes;
    const __amdgpu_buffer_rsrc_t ra = rsrc(a0 + k0, live ? rows_a * pitch - (int)k0 : 0);
    const __amdgpu_buffer_rsrc_t rb = rsrc(b0 + k0, live ? rows_b * pitch - (int)k0 : 0);
#pragma unroll
    for (int q = 0; q < QA; ++q) lds_dma<true>(ra, stage_a(S) + (wave + q * NW) * 256, off[q]);
#pragma unroll
    for (int q = 0; q < QB; ++q) lds_dma<true>(rb, stage_b(S) + (wave + q * NW) * 256, off[q]);
#pragma unroll
    for (int q = 0; q < QS; ++q) {
      const int u = wave + q * NW;  // uniform: which 64 rows of which granule
      const bool of_a = u < BM / 32;
      const int v = of_a ? u : u - BM / 32, per = of_a ? BM / 64 : BN / 64;
      const int g = 2 * t + v / per, r0 = v % per * 64;
      const unsigned *base = (of_a ? sa0 : sb0) + g * (of_a ? p.a.lds : p.b.lds);
      const int records = g < granules && u < US ? 4 * (of_a ? rows_a : rows_b) : 0;
      lds_dma<false>(rsrc(base, records), stage_s(S) + u * 64, (unsigned)(r0 + lane) * 4u);
    }
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

  Ops cur, nxt;
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
  // Slice t is in stage S, slices t + 1 .. t + NST - 1 on their way to the
  // others.  The last step waits for slice t + 1, and for every wave to be done
  // with stage S, then sends slice t + NST there and reads slice t + 1's first
  // operands.
  auto slice = [&](auto S, int t) {
    using SN = std::integral_constant<int, (decltype(S)::value + 1) % NST>;
    static_for<4>([&](auto STEP) {
      constexpr int s = decltype(STEP)::value;
      if constexpr (s < 3) {
        read_ops(S, s + 1, nxt);
        mma(STEP, cur);
        interleave(std::false_type());
      } else {
        dma_barrier_keep<(NST - 2) * kLoads>();
        dma(S, t + NST);
        read_ops(SN(), 0, nxt);
        read_scales(SN(), sn);
        mma(STEP, cur);
        interleave(std::true_type());
      }
      cur = nxt;
    });
    sc = sn;
  };

  if (nk > 0) {
    static_for<NST>([&](auto S) { dma(S, decltype(S)::value); });
    dma_barrier_keep<(NST - 1) * kLoads>();
    read_ops(S0(), 0, cur);
    read_scales(S0(), sc);
    for (int t = 0; t < nk; t += NST) {
      static_for<NST>([&](auto S) {
        if (decltype(S)::value == 0 || t + decltype(S)::value < nk) slice(S, t + decltype(S)::value);
      });
    }
    // The last slices sent loads past K (no memory traffic): let them retire
    // before the work-group gives up its LDS.
    __builtin_amdgcn_s_waitcnt(0x0f70);
  }

  // Register e of lane l holds row acc32_row(l, e), column l % 32 of a block:
  // row 4 (l / 32) of a uniform base and a constant number of rows past it.
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

template <int BM, int BN, int WM, int WN, int NST>
hipError_t launch(const Mxfp4Args &p, bool c_bf16, hipStream_t s) {
  const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  const long rows = p.offsets ? group_tile_rows(p.M, p.groups, BM) : tiles_m;
  const dim3 grid((unsigned)(rows * tiles_n)), block(WM * WN * kWave);
  const TileMap tmap = make_tile_map(tiles_m, tiles_n, 8);
  if (c_bf16)
    hipLaunchKernelGGL((mxfp4_tile_kernel<BM, BN, WM, WN, NST, true>), grid, block, 0, s, p, tmap,
                       tiles_n);
  else
    hipLaunchKernelGGL((mxfp4_tile_kernel<BM, BN, WM, WN, NST, false>), grid, block, 0, s, p, tmap,
                       tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_tile(int tile, const Mxfp4Args &p, bool c_bf16, hipStream_t s) {
  return tile == 256 ? launch<256, 256, 2, 4, 2>(p, c_bf16, s)
                     : launch<128, 128, 2, 2, 2>(p, c_bf16, s);
}

}  // namespace sgemm
