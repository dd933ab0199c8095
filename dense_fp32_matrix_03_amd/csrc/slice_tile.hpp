// slice_tile.hpp -- the main loop of a tile of A B^T whose operand slices of 128
// bytes a row reach LDS by buffer-to-LDS loads, for the formats of 8-bit integers
// (int8_tile.hip) and of numbers split into two half-precision pieces
// (orthogonalize.hip).
//
// A slice is [row][8 chunks of 16 bytes] in LDS, chunk c at c ^ kc_swizzle
// (mfma_dma.hpp), which is conflict-free for 16 lanes that read one chunk of 16
// consecutive rows.  There are two stages: while one is multiplied the other is
// loaded.  The descriptors end at the last row's last byte, so rows past it read
// as zeros.
//
// A format F gives
//   Acc              16 sums of a lane's block of 32 x 32, 4 bytes each
//   kSteps           steps of a slice
//   Frag             a lane's operands of 32 rows in a step
//   load(row, at)    reads a Frag from LDS: `at` gives the address of a chunk
//   kReads           its LDS reads
//   mma(a, b, acc)   a step's products; kMfma matrix instructions.
#pragma once

#include "mfma_dma.hpp"

namespace sgemm {

typedef int slice_i32x4 __attribute__((ext_vector_type(4)));

constexpr int kSliceRow = 128;  // bytes of a row's slice

// KS sets of WM x WN waves share a tile; set q takes slices q, q + KS, ..
// through LDS stages of its own, and the sets' sums are added in order at the
// end.  With few tiles the time is a chain of slices, each as long as its
// loads take to arrive: the sets walk KS chains at once.
template <class F, int BM, int BN, int WM, int WN, int KS>
struct SliceTile {
  static constexpr int NW = WM * WN;  // waves of a set
  static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  static constexpr int kThreads = NW * KS * kWave;
  static constexpr int QA = BM * kSliceRow / 1024 / NW, QB = BN * kSliceRow / 1024 / NW;
  static_assert(QA * NW * 1024 == BM * kSliceRow && QB * NW * 1024 == BN * kSliceRow,
                "loads must split evenly over the waves");
  static constexpr int kLoads = QA + QB;
  using Acc = typename F::Acc;
  using Word = decltype(Acc()[0] + Acc()[0]);

  // Where this wave's sums lie in the tile.
  __device__ __forceinline__ static int wave_id() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) % NW;
  }
  __device__ __forceinline__ static int row0() { return wave_id() / WN * WTM; }
  __device__ __forceinline__ static int col0() { return wave_id() % WN * WTN; }

  // acc = the tile's sums over nk slices.  a, b: the first rows' first bytes, rows
  // a_pitch (b_pitch) bytes apart, at least 128 nk; rows_a (rows_b) of them are
  // there.  BM a_pitch and BN b_pitch stay below 2^31.  False for waves
  // whose sums went to another set.
  __device__ __forceinline__ static bool run(const char *a, int a_pitch, int rows_a, const char *b,
                                             int b_pitch, int rows_b, int nk,
                                             Acc (&acc)[FM][FN]) {
    // One LDS array per stage and operand, so that the compiler sees that loads
    // into one stage do not touch the one that is read (mfma_dma.hpp).
    constexpr int SA = BM * kSliceRow / 4, SB = BN * kSliceRow / 4;
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

    // Load q of a wave fetches rows 8 (wave + q NW) .. + 7 of the slice.
    unsigned off_a[QA], off_b[QB];
    auto offset = [&](int q, int pitch) {
      const int row = 8 * (wave + q * NW) + lane / 8;
      return (unsigned)(row * pitch + 16 * ((lane % 8) ^ kc_swizzle<32, true>(row)));
    };
#pragma unroll
    for (int q = 0; q < QA; ++q) off_a[q] = offset(q, a_pitch);
#pragma unroll
    for (int q = 0; q < QB; ++q) off_b[q] = offset(q, b_pitch);

    auto rsrc = [](const void *base, int records) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, records,
                                               kRawBufferWord3);
    };
    // Loads of the set's next slice into stage S.  Slices at or past nk get
    // descriptors without records: nothing is fetched.  No branch depends on
    // that, so that the loads can be scheduled between matrix-core instructions.
    int k = kq;  // the slice
    auto dma = [&](auto S) {
      const bool live = k < nk;
      const int k0 = k * kSliceRow;
      const __amdgpu_buffer_rsrc_t ra = rsrc(a + k0, live ? rows_a * a_pitch - k0 : 0);
      const __amdgpu_buffer_rsrc_t rb = rsrc(b + k0, live ? rows_b * b_pitch - k0 : 0);
#pragma unroll
      for (int q = 0; q < QA; ++q) lds_dma<true>(ra, stage_a(S) + (wave + q * NW) * 256, off_a[q]);
#pragma unroll
      for (int q = 0; q < QB; ++q) lds_dma<true>(rb, stage_b(S) + (wave + q * NW) * 256, off_b[q]);
      k += KS;
    };

    const int sw = kc_swizzle<32, true>(r32);
    struct Ops {
      typename F::Frag a[FM], b[FN];
    };
    auto read_ops = [&](auto S, auto STEP, Ops &o) {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float *row = stage_a(S) + (wm * WTM + i * 32 + r32) * 32;
        o.a[i] = F::template load<decltype(STEP)::value>(
            half, [&](int c) { return reinterpret_cast<const slice_i32x4 *>(row + (c ^ sw) * 4); });
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const float *row = stage_b(S) + (wn * WTN + j * 32 + r32) * 32;
        o.b[j] = F::template load<decltype(STEP)::value>(
            half, [&](int c) { return reinterpret_cast<const slice_i32x4 *>(row + (c ^ sw) * 4); });
      }
    };

#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

    auto mma = [&](const Ops &o) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) F::mma(o.a[i], o.b[j], acc[i][j]);
    };

    // A step's operand reads (and a slice's loads) are spread between its
    // matrix-core instructions.
    constexpr int kMfma = FM * FN * F::kMfma, kReads = (FM + FN) * F::kReads;
    auto interleave = [&](auto last) {
      constexpr int loads = decltype(last)::value ? kLoads : 0;
      static_for<kMfma>([&](auto I) {
        constexpr int i = decltype(I)::value;
        constexpr int v = loads * (i + 1) / kMfma - loads * i / kMfma;
        constexpr int d = kReads * (i + 1) / kMfma - kReads * i / kMfma;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // matrix core
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
    constexpr int kSteps = F::kSteps, kAhead = WHOLE ? kSteps : 1;
    Ops cur[kAhead], nxt[kAhead];
    auto read_ahead = [&](auto S, Ops *o) {
      static_for<kAhead>([&](auto STEP) { read_ops(S, STEP, o[decltype(STEP)::value]); });
    };
    auto slice = [&](auto S) {
      using SN = std::integral_constant<int, 1 - decltype(S)::value>;
      if constexpr (WHOLE) {
        dma_barrier_keep<0>();
        dma(S);
        read_ahead(SN(), nxt);
        static_for<kSteps>([&](auto STEP) { mma(cur[decltype(STEP)::value]); });
#pragma unroll
        for (int s = 0; s < kAhead; ++s) cur[s] = nxt[s];
      } else {
        static_for<kSteps>([&](auto STEP) {
          constexpr int s = decltype(STEP)::value;
          if constexpr (s < kSteps - 1) {
            read_ops(S, std::integral_constant<int, s + 1>(), nxt[0]);
            mma(cur[0]);
            interleave(std::false_type());
          } else {
            dma_barrier_keep<0>();
            dma(S);
            read_ops(SN(), S0(), nxt[0]);
            mma(cur[0]);
            interleave(std::true_type());
          }
          cur[0] = nxt[0];
        });
      }
    };

    if (nk > 0) {
      const int turns = (nk + KS - 1) / KS;  // the same for all sets: they share the barriers
      dma(S0());
      dma(S1());
      dma_barrier_keep<kLoads>();
      read_ahead(S0(), cur);
      for (int t = 0; t < turns; t += 2) {
        slice(S0());
        if (t + 1 < turns) slice(S1());
      }
      // The last slices sent loads past the end (no memory traffic): let them
      // retire before the work-group gives up its LDS.
      __builtin_amdgcn_s_waitcnt(0x0f70);
    }

    if constexpr (KS > 1) {
      // The stages are free: every load has landed, every operand has been read.
      // Set s > 0 leaves its sums at 4 Ki (s - 1) of As0, the last of four sets in
      // Bs0.
      static_assert(FM * FN * NW == 4 && (KS == 2 || KS == 4) && KS * SA == 2048 * KS &&
                        SB == SA, "a set's sums are 16 KiB");
      __syncthreads();
      auto sums = [&](int set) {
        return reinterpret_cast<Word *>(set == 3 ? Bs0 : As0 + (set - 1) * 4096) + wave * 1024 +
               lane;
      };
      if (kq > 0) {
        Word *at = sums(kq);
#pragma unroll
        for (int e = 0; e < 16; ++e) at[e * kWave] = acc[0][0][e];
      }
      __syncthreads();
      if (kq > 0) return false;
#pragma unroll
      for (int set = 1; set < KS; ++set)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[0][0][e] += sums(set)[e * kWave];
    }
    return true;
  }
};

}  // namespace sgemm
