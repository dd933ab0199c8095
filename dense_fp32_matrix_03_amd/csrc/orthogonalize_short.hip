// orthogonalize_short.hip -- Newton-Schulz steps on matrices whose shorter side is at
// most 64 (include/sgemm_orthogonalize.h), in single precision on
// v_mfma_f32_32x32x2_f32.
//
// Such matrices (of adapters of low rank, of small heads) have so little work that
// launches decide: orthogonalize.hip takes three for a step, here it is one.  A
// work-group has a slab of columns of Z, 64 at a time.  It adds up the slabs' parts of S
// = Z Z^T, in their order, makes P = b S + c S S (each work-group for itself), Z = a Z +
// P Z for its columns, and its part of the next S from them.
//
// Bound by what follows one another in a launch: the parts of S, then three chains of 32
// matrix instructions for each 64 columns.  Five steps, here and with the tiles of
// orthogonalize.hip: 64 x 64 53 and 67 us, 64 x 512 61 and 80, 64 x 2048 87 and 112,
// 32 x 4096 116 and 145, 32 of 64 x 4096 225 and 262, 8 of 20 x 1000 67 and 83; only very
// many tiny ones lose (4000 of 64 x 1 470 and 451).
#include "orthogonalize.hpp"

namespace sgemm {

namespace {

constexpr int kThreads = 256;

// 64 x 64 floats, rows 65 apart: lanes that read a column fall on distinct banks.
struct Square {
  float at[64][65];
};

// The sum of k < 64 of A(r0 + r, k) B(k, c0 + c), a block of 32 x 32 per wave, to which
// acc is added; B transposed: B(c0 + c, k).
template <bool TB>
__device__ __forceinline__ void multiply(const Square &A, int r0, const Square &B, int c0,
                                         f32x16 &acc) {
  const int r32 = threadIdx.x % 32, half = threadIdx.x % kWave / 32;
#pragma unroll 8
  for (int k = 0; k < 64; k += 2) {
    const float a = A.at[r0 + r32][k + half];
    const float b = TB ? B.at[c0 + r32][k + half] : B.at[k + half][c0 + r32];
    acc = mfma32x32x2(a, b, acc);
  }
}

// Columns c0 .. c0 + 63 of a matrix to registers, from there (zeros past it) to a square,
// and from a square to memory.  Neighbouring threads have neighbouring elements of memory.
template <class T>
__device__ __forceinline__ void load_square(const T *x, long rs, long cs, int m, int n, int c0,
                                            float v[16]) {
  const bool along = cs == 1;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int slow = threadIdx.x / 64 + 4 * i, fast = threadIdx.x % 64;
    const int r = along ? slow : fast, c = c0 + (along ? fast : slow);
    v[i] = (float)x[min(r, m - 1) * rs + (long)min(c, n - 1) * cs];
  }
}
__device__ __forceinline__ void put_square(const float v[16], long cs, int m, int n, int c0,
                                           double scale, Square &to) {
  const bool along = cs == 1;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int slow = threadIdx.x / 64 + 4 * i, fast = threadIdx.x % 64;
    const int r = along ? slow : fast, c = along ? fast : slow;
    to.at[r][c] = r < m && c0 + c < n ? (float)(scale * (double)v[i]) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store_square(T *y, long rs, long cs, int m, int n, int c0,
                                             float scale, const Square &from) {
  const bool along = cs == 1;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int slow = threadIdx.x / 64 + 4 * i, fast = threadIdx.x % 64;
    const int r = along ? slow : fast, c = along ? fast : slow;
    if (r < m && c0 + c < n) y[r * rs + (long)(c0 + c) * cs] = (T)(scale * from.at[r][c]);
  }
}

__device__ __forceinline__ double group_sum(double v) {
  __shared__ double part[kThreads / kWave];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  return part[0] + part[1] + part[2] + part[3];
}

// FIRST: Z = X / (|X| + eps), and S's part.  Else a step; LAST: to Y, without a part.
template <bool FIRST, bool LAST, class T>
__global__ void __launch_bounds__(kThreads) ortho_short_kernel(OrthoShortArgs p) {
  __shared__ Square z, s, q;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int slab = blockIdx.x, batch = blockIdx.y;
  const int r0 = wave / 2 * 32, c32 = wave % 2 * 32;  // the wave's block of a square
  const int m = p.m, n = p.n;
  const long zs = (long)m * n;
  double scale = 1.0;
  float next[16];  // the next 64 columns
  auto load_next = [&](int c0) {
    if constexpr (FIRST)
      load_square(static_cast<const T *>(p.X) + batch * p.strideX, p.xr, p.xc, m, n, c0, next);
    else
      load_square(p.z_in + batch * zs, (long)n, 1L, m, n, c0, next);
  };
  load_next(slab * p.blocks * 64);
  if constexpr (FIRST) {
    const double part = (int)threadIdx.x < p.norm.n_parts
                            ? p.norm.parts[(long)batch * p.norm.n_parts + threadIdx.x] : 0.0;
    const double norm = sqrt(group_sum(part)) + (double)p.eps;
    scale = norm > 0 ? 1.0 / norm : norm;  // NaN stays
  } else {
    // S: 16 elements a thread, of four slabs together.
    float sum[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] = 0.f;
    const float *const parts = p.part_in + (long)batch * p.slabs * m * m;
    for (int k = 0; k < p.slabs; k += 4) {
      float v[4][16];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[j][i] = parts[(long)min(k + j, p.slabs - 1) * m * m +
                          min((int)threadIdx.x + i * kThreads, m * m - 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] += k + j < p.slabs ? v[j][i] : 0.f;
    }
    for (int i = threadIdx.x; i < 64 * 64; i += kThreads) s.at[i / 64][i % 64] = 0.f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = threadIdx.x + i * kThreads, r = p.by_m(at);
      if (at < m * m) s.at[r][at - r * m] = sum[i];
    }
    __syncthreads();
    f32x16 acc = {};
    multiply<true>(s, r0, s, c32, acc);  // S is symmetric
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int r = r0 + acc32_row(lane, e), c = c32 + lane % 32;
      q.at[r][c] = fmaf(p.b, s.at[r][c], p.c * acc[e]);
    }
    __syncthreads();
  }
  f32x16 part = {};
  for (int block = 0; block < p.blocks; ++block) {
    const int c0 = (slab * p.blocks + block) * 64;
    if (c0 >= n) break;
    if (block > 0) __syncthreads();  // the last block's reads of z
    put_square(next, FIRST ? p.xc : 1L, m, n, c0, scale, z);
    if (block + 1 < p.blocks) load_next(c0 + 64);
    __syncthreads();
    if constexpr (!FIRST) {
      f32x16 acc = {};
      multiply<false>(q, r0, z, c32, acc);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[e] = fmaf(p.a, z.at[r0 + acc32_row(lane, e)][c32 + lane % 32], acc[e]);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 16; ++e) z.at[r0 + acc32_row(lane, e)][c32 + lane % 32] = acc[e];
      __syncthreads();
    }
    if constexpr (LAST) {
      store_square(static_cast<T *>(p.Y) + batch * p.strideY, p.yr, p.yc, m, n, c0, p.alpha, z);
    } else {
      store_square(p.z_out + batch * zs, (long)n, 1L, m, n, c0, 1.f, z);
      multiply<true>(z, r0, z, c32, part);
    }
  }
  if constexpr (!LAST) {
    float *const to = p.part_out + ((long)batch * p.slabs + slab) * m * m;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int r = r0 + acc32_row(lane, e), c = c32 + lane % 32;
      if (r < m && c < m) to[r * m + c] = part[e];
    }
  }
}

}  // namespace

hipError_t launch_ortho_short(const OrthoShortArgs &p, bool first, bool last, bool bf16, int batch,
                              hipStream_t s) {
  const dim3 grid((unsigned)p.slabs, (unsigned)batch), block(kThreads);
  if (first) {
    if (bf16)
      hipLaunchKernelGGL((ortho_short_kernel<true, false, __bf16>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((ortho_short_kernel<true, false, float>), grid, block, 0, s, p);
  } else if (last) {
    if (bf16)
      hipLaunchKernelGGL((ortho_short_kernel<false, true, __bf16>), grid, block, 0, s, p);
    else
      hipLaunchKernelGGL((ortho_short_kernel<false, true, float>), grid, block, 0, s, p);
  } else {
    hipLaunchKernelGGL((ortho_short_kernel<false, false, float>), grid, block, 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace sgemm
