// slice_tile.hpp -- the main loop of a tile of A B^T whose operand slices of 128
// bytes a row reach LDS by buffer-to-LDS loads, for the formats of 8-bit integers
// (int8_tile.hip) and of numbers split into two half-precision pieces
// (orthogonalize.hip).
//
// A slice is [row][8 chunks of 16 bytes] in LDS, chunk c at c ^ kc_swizzle
// (mfma_dma.hpp), which is conflict-free for 16 lanes that read one chunk of 16
// consecutive rows.  There are NST stages: while one is multiplied the others are
// loaded.  The descriptors end at the last row's last byte, so rows past it read
// as zeros.
//
// A format F gives
//   Acc              16 sums of a lane's block of 32 x 32, 4 bytes each
//   kSteps           steps of a slice
//   Frag             a lane's operands of 32 rows in a step
//   load(row, at)    reads a Frag from LDS: `at` gives the address of a chunk
//   kReads           its LDS reads
//   mma<I>(a, b, acc)  the I-th of the kMfma matrix instructions of a step.
// An instruction that adds to the sums of the one before waits for it: the
// instructions of a step go through all blocks one by one, and a wave with a single
// block adds to kChains sums in turn.
#pragma once

#include "mfma_dma.hpp"

namespace sgemm {

typedef int slice_i32x4 __attribute__((ext_vector_type(4)));

constexpr int kSliceRow = 128;  // bytes of a row's slice

// Barrier of the work-group that retires all except this wave's N most recent
// buffer-to-LDS loads, and its LDS reads and writes.  __syncthreads is a fence too, at
// which the compiler waits for every such load, so that no more than one slice was
// ever on its way, however many stages there were.  Here the waits are the ones
// written (s_waitcnt: vmcnt(N), lgkmcnt(0)), and the fences of a single wave only
// keep the compiler from moving LDS accesses across.
template <int N>
__device__ __forceinline__ void slice_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_s_waitcnt((N & 15) | (0x7 << 4) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Rows of an operand: the first one's first slice, and the bytes from a row and from
// a slice to the next (row_step x the tile's rows stays below 2^31).  Rows one after
// the other have row_step = their length and slice_step = 128.  Where that length is
// a multiple of some KiB, the slices that the whole chip reads at a time lie in few
// of the memory's channels: 8192^3 in 8-bit integers 540 us with both operands' rows
// 8192 bytes apart, 459 with rows 8320 apart.  Slices one after the other, row_step =
// 128, are free of that.
struct SliceRows {
  const char *at;
  int row_step;
  long slice_step;
  int rows;
  // The same in scalar registers.  All waves of a work-group have the same operands,
  // but where the compiler does not see it, as with tiles of groups, it wraps each
  // load in a loop over the lanes' descriptors.
  __device__ __forceinline__ SliceRows uniform() const {
    auto u32 = [](unsigned v) { return (unsigned)__builtin_amdgcn_readfirstlane((int)v); };
    auto u64 = [&](uint64_t v) {
      return (uint64_t)u32((unsigned)(v >> 32)) << 32 | u32((unsigned)v);
    };
    return {reinterpret_cast<const char *>(u64(reinterpret_cast<uint64_t>(at))),
            (int)u32((unsigned)row_step), (long)u64((uint64_t)slice_step), (int)u32((unsigned)rows)};
  }
};

// WM x WN waves have a tile of BM x BN.
template <class F, int BM, int BN, int WM, int WN, int NST>
struct SliceTile {
  static constexpr int NW = WM * WN;  // waves
  static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  static constexpr int kThreads = NW * kWave;
  static constexpr int QA = BM * kSliceRow / 1024 / NW, QB = BN * kSliceRow / 1024 / NW;
  static_assert(QA * NW * 1024 == BM * kSliceRow && QB * NW * 1024 == BN * kSliceRow,
                "loads must split evenly over the waves");
  static constexpr int kLoads = QA + QB;
  using Acc = typename F::Acc;

  // Where this wave's sums lie in the tile.
  __device__ __forceinline__ static int wave_id() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  }
  __device__ __forceinline__ static int row0() { return wave_id() / WN * WTM; }
  __device__ __forceinline__ static int col0() { return wave_id() % WN * WTN; }

  // acc = the tile's sums over nk slices.  lds: the stages' memory (STAGE_BYTES each),
  // free once all waves have passed another barrier.  meanwhile(): work for the time that
  // the first slices take, before the first of run's barriers (where nk > 0).
  static constexpr int STAGE_BYTES = (BM + BN) * kSliceRow;
  struct Nothing {
    __device__ __forceinline__ void operator()() const {}
  };
  template <class Meanwhile = Nothing>
  __device__ __forceinline__ static void run(const SliceRows &rows_a, const SliceRows &rows_b,
                                             int nk, Acc (&acc)[FM][FN], char *(&lds)[NST],
                                             const Meanwhile &meanwhile = Meanwhile()) {
    const SliceRows a = rows_a.uniform(), b = rows_b.uniform();
    // One LDS array per stage, so that the compiler sees that loads into one stage do
    // not touch the one that is read (mfma_dma.hpp).  It tells four arrays apart; with
    // one for each operand of four stages it waited for all loads before most reads.
    constexpr int SA = BM * kSliceRow / 4, SB = BN * kSliceRow / 4;
    static_assert(NST >= 2 && NST <= 4, "two to four stages");
    constexpr auto room = [](int stage) { return stage < NST ? SA + SB : 4; };
    __shared__ __attribute__((aligned(1024))) float stage0[room(0)], stage1[room(1)];
    __shared__ __attribute__((aligned(16))) float stage2[room(2)], stage3[room(3)];

    {
      float *const all[] = {stage0, stage1, stage2, stage3};
      for (int i = 0; i < NST; ++i) lds[i] = reinterpret_cast<char *>(all[i]);
    }
    const int lane = threadIdx.x % kWave;
    const int wave = wave_id();
    const int wm = wave / WN, wn = wave % WN;
    const int r32 = lane % 32, half = lane / 32;
    // An address is the array and a single offset: through more steps than that the
    // compiler loses sight of the array.
    auto stage = [&](auto S) -> float * {
      constexpr int s = decltype(S)::value;
      return s == 0 ? stage0 : s == 1 ? stage1 : s == 2 ? stage2 : stage3;
    };

    // Load q of a wave fetches rows 8 (wave + q NW) .. + 7 of the slice.
    unsigned off_a[QA], off_b[QB];
    auto offset = [&](int q, int step) {
      const int row = 8 * (wave + q * NW) + lane / 8;
      return (unsigned)(row * step + 16 * ((lane % 8) ^ kc_swizzle<32, true>(row)));
    };
#pragma unroll
    for (int q = 0; q < QA; ++q) off_a[q] = offset(q, a.row_step);
#pragma unroll
    for (int q = 0; q < QB; ++q) off_b[q] = offset(q, b.row_step);

    auto rsrc = [](const void *base, int records) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, records,
                                               kRawBufferWord3);
    };
    // Loads of the next slice into stage S.  Slices at or past nk get
    // descriptors without records: nothing is fetched.  No branch depends on
    // that, so that the loads can be scheduled between matrix-core instructions.
    int k = 0;  // the slice
    const int end_a = (a.rows - 1) * a.row_step + kSliceRow;
    const int end_b = (b.rows - 1) * b.row_step + kSliceRow;
    auto dma = [&](auto S) {
      const bool live = k < nk;
      const __amdgpu_buffer_rsrc_t ra = rsrc(a.at + k * a.slice_step, live ? end_a : 0);
      const __amdgpu_buffer_rsrc_t rb = rsrc(b.at + k * b.slice_step, live ? end_b : 0);
#pragma unroll
      for (int q = 0; q < QA; ++q) lds_dma<true>(ra, stage(S) + (wave + q * NW) * 256, off_a[q]);
#pragma unroll
      for (int q = 0; q < QB; ++q) lds_dma<true>(rb, stage(S) + (SA + (wave + q * NW) * 256), off_b[q]);
      ++k;
    };

    const int sw = kc_swizzle<32, true>(r32);
    struct Ops {
      typename F::Frag a[FM], b[FN];
    };
    // B first: its operands are needed first.
    auto read_ops = [&](auto S, auto STEP, Ops &o) {
      auto read = [&](int row) {
        return F::template load<decltype(STEP)::value>(half, [&](int c) {
          return reinterpret_cast<const slice_i32x4 *>(stage(S) + (row + (c ^ sw) * 4));
        });
      };
#pragma unroll
      for (int j = 0; j < FN; ++j) o.b[j] = read(SA + (wn * WTN + j * 32 + r32) * 32);
#pragma unroll
      for (int i = 0; i < FM; ++i) o.a[i] = read((wm * WTM + i * 32 + r32) * 32);
    };

#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

    // The sums that a wave with one block adds to in turn, but for the last.
    constexpr int kChains = FM * FN == 1 ? F::kChains : 1;
    Acc chain[kChains];
#pragma unroll
    for (int c = 0; c + 1 < kChains; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) chain[c][e] = 0;
    auto mma = [&](auto STEP, const Ops &o) {
      static_for<F::kMfma>([&](auto I) {
        constexpr int c = (decltype(STEP)::value * F::kMfma + decltype(I)::value) % kChains;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            F::template mma<decltype(I)::value>(o.a[i], o.b[j],
                                                c + 1 < kChains ? chain[c] : acc[i][j]);
      });
    };

    // A step's operand reads (and a slice's loads) are spread between its
    // matrix-core instructions, the reads over the first three quarters of them: they
    // have arrived when the next step begins.
    constexpr int kMfma = FM * FN * F::kMfma, kReads = (FM + FN) * F::kReads;
    auto interleave = [&](auto steps, auto last) {  // of that many steps together
      constexpr int mfma = kMfma * decltype(steps)::value, reads = kReads * decltype(steps)::value;
      constexpr int loads = decltype(last)::value ? kLoads : 0;
      static_for<mfma>([&](auto I) {
        constexpr int i = decltype(I)::value;
        constexpr int v = loads * (i + 1) / mfma - loads * i / mfma;
        constexpr int span = (mfma * 3 + 3) / 4;
        constexpr int d = reads * (i + 1 < span ? i + 1 : span) / span -
                          reads * (i < span ? i : span) / span;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // matrix core
        if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);  // DS read
        if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);  // VMEM read
      });
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    // Slice t is in stage S, the next ones on their way to the others.
    // WHOLE: a wave with one block of 32 x 32 has too few matrix-core
    // instructions in a step to cover the next one's reads, and registers to
    // spare: it reads a whole slice's operands while it multiplies the one
    // before.  The barrier waits for slice t + 1, and for every wave to have read
    // slice t; then slice t + NST goes to stage S.
    // Otherwise the operands are read a step ahead, and the last step of a slice
    // waits for slice t + 1, and for every wave to be done with stage S, sends
    // slice t + NST there and reads slice t + 1's first operands.
    constexpr bool WHOLE = FM * FN == 1;
    constexpr int kSteps = F::kSteps, kAhead = WHOLE ? kSteps : 1;
    Ops cur[kAhead], nxt[kAhead];
    auto read_ahead = [&](auto S, Ops *o) {
      static_for<kAhead>([&](auto STEP) { read_ops(S, STEP, o[decltype(STEP)::value]); });
    };
    auto slice = [&](auto S) {
      using SN = std::integral_constant<int, (decltype(S)::value + 1) % NST>;
      if constexpr (WHOLE) {
        slice_barrier<(NST - 2) * kLoads>();
        dma(S);
        read_ahead(SN(), nxt);
        static_for<kSteps>([&](auto STEP) { mma(STEP, cur[decltype(STEP)::value]); });
        interleave(std::integral_constant<int, kSteps>(), std::true_type());
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < kAhead; ++s) cur[s] = nxt[s];
      } else {
        static_for<kSteps>([&](auto STEP) {
          constexpr int s = decltype(STEP)::value;
          if constexpr (s < kSteps - 1) {
            read_ops(S, std::integral_constant<int, s + 1>(), nxt[0]);
            mma(STEP, cur[0]);
            interleave(S1(), std::false_type());
          } else {
            slice_barrier<(NST - 2) * kLoads>();
            dma(S);
            read_ops(SN(), S0(), nxt[0]);
            mma(STEP, cur[0]);
            interleave(S1(), std::true_type());
          }
          cur[0] = nxt[0];
        });
      }
    };

    if (nk > 0) {
      static_for<NST>([&](auto S) { dma(S); });
      meanwhile();
      slice_barrier<(NST - 1) * kLoads>();
      read_ahead(S0(), cur);
      // Whole rounds of the stages without a test between them, then the rest: at a
      // branch the compiler would lose count of the loads on their way.
      int t = 0;
      for (; t + NST <= nk; t += NST) static_for<NST>([&](auto S) { slice(S); });
      static_for<NST - 1>([&](auto S) {
        if (t + decltype(S)::value < nk) slice(S);
      });
      // The last slices sent loads past the end (no memory traffic): let them
      // retire before the work-group gives up its LDS.
      __builtin_amdgcn_s_waitcnt(0x0f70);
    }

#pragma unroll
    for (int c = 0; c + 1 < kChains; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[0][0][e] += chain[c][e];
  }
};

}  // namespace sgemm
