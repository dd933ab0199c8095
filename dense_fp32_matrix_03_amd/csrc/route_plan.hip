// route_plan.hip -- pairs of tokens and picks sorted by expert
// (sgemm_route_plan in include/sgemm_route.h).
//
// A counting sort that keeps the pairs' order inside a group.  A chunk of
// consecutive pairs has a work-group.  A first launch counts each chunk's pairs
// by group (left out where there is one chunk); a second one sums the counts
// before its chunk and places its pairs: each wave has a quarter of the chunk and
// takes it 64 pairs at a time, a pair's place being that of its group so far
// and the number of lanes before it with the same group, which ballots over the
// bits of the group's number give.  Nothing depends on the order of atomics:
// they only count.
//
// Held by trips to memory, one after the other: picks, counts, places; 12 bytes a pair
// would take 0.2 us for 65536 pairs.  So a lane loads up to 8 picks, and 16 chunks'
// counts, together.  By graph replay: 48 pairs of 16 groups 3.1 us; 65536 of 128 groups
// 10.7 us (23.5 with one load at a time and chunks of 4096 pairs, 15.0 with 16 picks
// together and those chunks, but then 4.3 for 48 pairs, whose code is longer); 131072 of
// 1024 groups 22 us, 16384 of 4096 groups 27 us.
#include "route.hpp"

namespace sgemm {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;

// The groups of pairs at + i * step + lane below `end` for i < H, or -1.  `at` and `end`
// are the same for a wave.
template <int H>
__device__ __forceinline__ void load_groups(const PlanArgs &p, long at, int step, long end,
                                            int g[H]) {
  const int lane = threadIdx.x % kWave;
  int pick[H];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    pick[i] = 0;
    if (at + i * step < end) pick[i] = p.picks[min(at + i * step + lane, end - 1)];
  }
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const long own = (long)pick[i] - p.first;
    g[i] = at + i * step + lane < end && own >= 0 && own < p.groups ? (int)own : -1;
  }
}

// G: groups that there is room for.  H: pairs of a lane whose picks are loaded together.
template <int G, int H>
__global__ void __launch_bounds__(kThreads) plan_count_kernel(PlanArgs p) {
  __shared__ int count[G];
  for (int g = threadIdx.x; g < p.groups; g += kThreads) count[g] = 0;
  __syncthreads();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const long begin = (long)blockIdx.x * p.chunk, end = min(begin + p.chunk, (long)p.pairs);
  for (long at = begin + wave * kWave; at < end; at += kThreads * H) {
    int g[H];
    load_groups<H>(p, at, kThreads, end, g);
#pragma unroll
    for (int i = 0; i < H; ++i)
      if (g[i] >= 0) atomicAdd(&count[g[i]], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < p.groups; g += kThreads)
    p.counts[(long)blockIdx.x * p.groups + g] = count[g];
}

template <int G, int H>
__global__ void __launch_bounds__(kThreads) plan_place_kernel(PlanArgs p) {
  __shared__ int next[kWaves * G];  // [waves][groups]: counts, then the next places
  __shared__ int base[G];           // totals, then the groups' first rows
  __shared__ int part[kThreads];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = blockIdx.x;
  const long begin = (long)c * p.chunk, end = min(begin + p.chunk, (long)p.pairs);
  const int quarter = p.chunk / kWaves;
  const long from = min(begin + wave * quarter, end), to = min(from + quarter, end);
  constexpr int kStep = kWave * H;

  int held[H];
  load_groups<H>(p, from, kWave, to, held);
  for (int i = tid; i < kWaves * p.groups; i += kThreads) next[i] = 0;
  __syncthreads();
  for (long at = from;;) {
#pragma unroll
    for (int i = 0; i < H; ++i)
      if (held[i] >= 0) atomicAdd(&next[wave * p.groups + held[i]], 1);
    at += kStep;
    if (at >= to) break;
    load_groups<H>(p, at, kWave, to, held);
  }
  __syncthreads();

  // Each group's total over all chunks, and where this chunk's waves place theirs, so
  // far from the group's first row.
  for (int g = tid; g < p.groups; g += kThreads) {
    int total = 0, before = 0;
    if (p.chunks > 1) {
      constexpr int kTogether = 16;
      for (int k = 0; k < p.chunks; k += kTogether) {
        int n[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          n[j] = p.counts[(long)min(k + j, p.chunks - 1) * p.groups + g];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
          before += k + j < c ? n[j] : 0;
          total += k + j < p.chunks ? n[j] : 0;
        }
      }
    }
    int at = before;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int n = next[w * p.groups + g];
      next[w * p.groups + g] = at;
      at += n;
    }
    base[g] = p.chunks > 1 ? total : at;
  }
  __syncthreads();

  // The groups' first rows: each thread has `per` consecutive groups, and a scan over
  // the threads gives the rows before them.
  const int per = (p.groups + kThreads - 1) / kThreads;
  int mine = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < p.groups) mine += base[tid * per + i];
  part[tid] = mine;
  __syncthreads();
  for (int d = 1; d < kThreads; d *= 2) {
    const int v = tid >= d ? part[tid - d] : 0;
    __syncthreads();
    part[tid] += v;
    __syncthreads();
  }
  int first = part[tid] - mine;
  const int all = part[kThreads - 1];
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    if (g >= p.groups) break;
    const int total = base[g];
    base[g] = first;
    if (c == 0) p.offsets[g] = first;
    first += total;
  }
  if (c == 0 && tid == 0) p.offsets[p.groups] = all;
  __syncthreads();

  const int bits = p.groups > 1 ? 32 - __builtin_clz(p.groups - 1) : 0;
  for (long at = from; at < to; at += kStep) {
    if (to - from > kStep) load_groups<H>(p, at, kWave, to, held);
#pragma unroll
    for (int k = 0; k < H; ++k) {
      if (at + k * kWave >= to) break;
      const long i = at + k * kWave + lane;
      const int g = held[k];
      unsigned long long same = __ballot(g >= 0);
      for (int b = 0; b < bits; ++b) {
        const bool bit = g >> b & 1;
        const unsigned long long ones = __ballot(bit);
        same &= bit ? ones : ~ones;
      }
      if (g >= 0) {
        const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32),
                                                     __builtin_amdgcn_mbcnt_lo((unsigned)same, 0));
        const int at_g = next[wave * p.groups + g];
        const int place = base[g] + at_g + before;
        p.places[i] = place;
        p.sources[place] = (int)i;
        // Every lane of the group has read the count by now; its last one moves it on.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (before == __builtin_popcountll(same) - 1)
          next[wave * p.groups + g] = at_g + before + 1;
      } else if (i < to) {
        p.places[i] = -1;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  for (long r = begin + tid; r < end; r += kThreads)
    if (r >= all) p.sources[r] = -1;
}

template <int G, int H>
hipError_t launch(const PlanArgs &p, hipStream_t s) {
  const dim3 grid((unsigned)p.chunks), block(kThreads);
  if constexpr (H > 1)  // one load a lane: one chunk
    if (p.chunks > 1) {
      hipLaunchKernelGGL((plan_count_kernel<G, H>), grid, block, 0, s, p);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
  hipLaunchKernelGGL((plan_place_kernel<G, H>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_plan(const PlanArgs &p, hipStream_t s) {
  if (p.groups > 512) return launch<4096, 8>(p, s);
  // A chunk of 256 pairs is one load a lane.
  return p.chunk <= kThreads ? launch<512, 1>(p, s) : launch<512, 8>(p, s);
}

}  // namespace sgemm
