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
#include "route.hpp"

namespace sgemm {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;

// The group of a pair, or -1.
__device__ __forceinline__ int group_of(const PlanArgs &p, int pair) {
  const long g = (long)p.picks[pair] - p.first;
  return g >= 0 && g < p.groups ? (int)g : -1;
}

// G: groups that there is room for.
template <int G>
__global__ void __launch_bounds__(kThreads) plan_count_kernel(PlanArgs p) {
  __shared__ int count[G];
  for (int g = threadIdx.x; g < p.groups; g += kThreads) count[g] = 0;
  __syncthreads();
  const long begin = (long)blockIdx.x * p.chunk, end = min(begin + p.chunk, (long)p.pairs);
  for (long i = begin + threadIdx.x; i < end; i += kThreads) {
    const int g = group_of(p, (int)i);
    if (g >= 0) atomicAdd(&count[g], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < p.groups; g += kThreads)
    p.counts[(long)blockIdx.x * p.groups + g] = count[g];
}

template <int G>
__global__ void __launch_bounds__(kThreads) plan_place_kernel(PlanArgs p) {
  __shared__ int next[kWaves * G];  // [waves][groups]: counts, then the next places
  __shared__ int base[G];           // totals, then the groups' first rows
  __shared__ int part[kThreads];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int c = blockIdx.x;
  const long begin = (long)c * p.chunk, end = min(begin + p.chunk, (long)p.pairs);
  const long quarter = p.chunk / kWaves;
  const long from = min(begin + wave * quarter, end), to = min(from + quarter, end);

  for (int i = tid; i < kWaves * p.groups; i += kThreads) next[i] = 0;
  __syncthreads();
  for (long i = from + lane; i < to; i += kWave) {
    const int g = group_of(p, (int)i);
    if (g >= 0) atomicAdd(&next[wave * p.groups + g], 1);
  }
  __syncthreads();

  // Each thread has `per` consecutive groups: their totals over all chunks, and a
  // scan over the threads for the rows before them.
  const int per = (p.groups + kThreads - 1) / kThreads;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    if (g >= p.groups) break;
    int total = 0, before = 0;
    if (p.chunks > 1) {
      for (int k = 0; k < p.chunks; ++k) {
        const int n = p.counts[(long)k * p.groups + g];
        before += k < c ? n : 0;
        total += n;
      }
    } else {
      for (int w = 0; w < kWaves; ++w) total += next[w * p.groups + g];
    }
    base[g] = total;
    // The places in this chunk, so far from the group's first row.
    int at = before;
    for (int w = 0; w < kWaves; ++w) {
      const int n = next[w * p.groups + g];
      next[w * p.groups + g] = at;
      at += n;
    }
    mine += total;
  }
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
  for (long i0 = from; i0 < to; i0 += kWave) {
    const long i = i0 + lane;
    const int g = i < to ? group_of(p, (int)i) : -1;
    unsigned long long same = __ballot(g >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool bit = g >> b & 1;
      const unsigned long long ones = __ballot(bit);
      same &= bit ? ones : ~ones;
    }
    if (g >= 0) {
      const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((unsigned)same, 0));
      const int at = next[wave * p.groups + g];
      const int place = base[g] + at + before;
      p.places[i] = place;
      p.sources[place] = (int)i;
      // Every lane of the group has read the count by now; its last one moves it on.
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (before == __builtin_popcountll(same) - 1) next[wave * p.groups + g] = at + before + 1;
    } else if (i < to) {
      p.places[i] = -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  for (long r = begin + tid; r < end; r += kThreads)
    if (r >= all) p.sources[r] = -1;
}

template <int G>
hipError_t launch(const PlanArgs &p, hipStream_t s) {
  const dim3 grid((unsigned)p.chunks), block(kThreads);
  if (p.chunks > 1) {
    hipLaunchKernelGGL(plan_count_kernel<G>, grid, block, 0, s, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(plan_place_kernel<G>, grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_plan(const PlanArgs &p, hipStream_t s) {
  return p.groups <= 512 ? launch<512>(p, s) : launch<4096>(p, s);
}

}  // namespace sgemm
