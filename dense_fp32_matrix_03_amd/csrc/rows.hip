// rows.hip -- rows gathered by expert, brought back to their tokens, and the
// gradients of that (include/sgemm_route.h).
//
// Bound by memory.  A wave has a piece of up to 4096 bytes of a row, 16 bytes a
// lane in each of four loads that go out together.  8192 tokens, 8 rows each, 2048
// bfloat16 columns, operands not in the caches: combined in 61 us (302 MB, 4.9 TB/s, a
// large copy's rate); gathered in 76 (302 MB, nearly all of it written, 4.0 TB/s).
#include "piece.hpp"
#include "route.hpp"

namespace sgemm {

namespace {

constexpr int kUnits = 4;  // waves of a work-group

// The unit (row and piece of it) of a wave; false past the last.
__device__ __forceinline__ bool unit_of(const RowsArgs &p, long &row, int &piece) {
  const int u = blockIdx.x * kUnits + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = p.by_pieces(u);
  row = r;
  piece = u - r * p.pieces;
  return r < p.rows;
}

template <bool BF16>
__global__ void __launch_bounds__(kUnits *kWave) rows_gather_kernel(RowsArgs p) {
  using P = Piece<BF16>;
  long r;
  int piece;
  if (!unit_of(p, r, piece)) return;
  const int source = p.index[r];
  if (source < 0 || source >= p.limit) return;
  const int lane = threadIdx.x % kWave;
  const int n0 = piece * (kRowPiece / 16 * P::V) + lane * P::V;
  const bool whole = p.N - piece * (kRowPiece / 16 * P::V) >= kRowPiece / 16 * P::V;
  const long x = (long)(source / p.topk) * p.ldx, y = r * p.ldy;
  P v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + i * kWave * P::V;
    v[i].load(p.X, x + n, p.N - n, whole);
  }
  if (p.weights) {
    const float w = p.weights[source];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[P::V];
      v[i].get(f);
#pragma unroll
      for (int e = 0; e < P::V; ++e) f[e] *= w;
      v[i].set(f);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + i * kWave * P::V;
    v[i].store(p.Y, y + n, p.N - n);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kUnits *kWave) rows_combine_kernel(RowsArgs p) {
  using P = Piece<BF16>;
  long t;
  int piece;
  if (!unit_of(p, t, piece)) return;
  const int lane = threadIdx.x % kWave;
  const int n0 = piece * (kRowPiece / 16 * P::V) + lane * P::V;
  const bool whole = p.N - piece * (kRowPiece / 16 * P::V) >= kRowPiece / 16 * P::V;
  float sum[4][P::V];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < P::V; ++e) sum[i][e] = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    const long pair = t * p.topk + j;
    const int place = p.index[pair];
    if (place < 0 || place >= p.limit) continue;
    const float w = p.weights ? p.weights[pair] : 1.f;
    P v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + i * kWave * P::V;
      v[i].load(p.X, place * p.ldx + n, p.N - n, whole);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[P::V];
      v[i].get(f);
#pragma unroll
      for (int e = 0; e < P::V; ++e) sum[i][e] = fmaf(w, f[e], sum[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + i * kWave * P::V;
    P v;
    v.set(sum[i]);
    v.store(p.Y, t * p.ldy + n, p.N - n);
  }
}

// A wave has a pair, its whole row: the sum over columns needs no second launch.  1500
// tokens, 6 rows each, 777 single-precision columns, half of them held: 8.7 us, 10.3 with
// operands not in the caches (39 MB, 3.8 TB/s).
template <bool BF16>
__global__ void __launch_bounds__(kUnits *kWave) rows_combine_backward_kernel(RowsBackArgs p) {
  using P = Piece<BF16>;
  const long pair = (long)blockIdx.x * kUnits + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (pair >= p.pairs) return;
  const int lane = threadIdx.x % kWave;
  const int place = p.places[pair];
  if (place < 0 || place >= p.rows) {
    if (p.dweights && lane == 0) p.dweights[pair] = 0.f;
    return;
  }
  const long dy = pair / p.topk * p.lddy;
  const float w = p.weights ? p.weights[pair] : 1.f;
  float dot = 0.f;
  // Two steps' loads go out together.
  constexpr int kStep = kWave * P::V, kTogether = 2;
  for (int left = p.N; left > 0; left -= kTogether * kStep) {
    const int n0 = p.N - left + lane * P::V;
    P g[kTogether], x[kTogether];
    const bool whole = left >= kTogether * kStep;
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int n = n0 + i * kStep;
      g[i].load(p.dY, dy + n, p.N - n, whole);
      if (p.dweights) x[i].load(p.X, place * p.ldx + n, p.N - n, whole);
    }
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int n = n0 + i * kStep;
      float f[P::V], v[P::V];
      g[i].get(v);
      if (p.dweights) {
        x[i].get(f);
#pragma unroll
        for (int e = 0; e < P::V; ++e) dot = fmaf(f[e], v[e], dot);
      }
      if (p.dX) {
#pragma unroll
        for (int e = 0; e < P::V; ++e) v[e] *= w;
        g[i].set(v);
        g[i].store(p.dX, place * p.lddx + n, p.N - n);
      }
    }
  }
  if (p.dweights) {
#pragma unroll
    for (int d = 32; d > 0; d /= 2) dot += __shfl_xor(dot, d);
    if (lane == 0) p.dweights[pair] = dot;
  }
}

dim3 units(long n) { return dim3((unsigned)((n + kUnits - 1) / kUnits)); }

}  // namespace

hipError_t launch_rows_gather(const RowsArgs &p, bool bf16, hipStream_t s) {
  const dim3 grid = units((long)p.rows * p.pieces), block(kUnits * kWave);
  if (bf16)
    hipLaunchKernelGGL(rows_gather_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(rows_gather_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_rows_combine(const RowsArgs &p, bool bf16, hipStream_t s) {
  const dim3 grid = units((long)p.rows * p.pieces), block(kUnits * kWave);
  if (bf16)
    hipLaunchKernelGGL(rows_combine_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(rows_combine_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_rows_combine_backward(const RowsBackArgs &p, bool bf16, hipStream_t s) {
  const dim3 grid = units(p.pairs), block(kUnits * kWave);
  if (bf16)
    hipLaunchKernelGGL(rows_combine_backward_kernel<true>, grid, block, 0, s, p);
  else
    hipLaunchKernelGGL(rows_combine_backward_kernel<false>, grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace sgemm
