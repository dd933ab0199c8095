// grouped.hpp -- launchers of the products whose rows fall into groups
// (grouped.hip), and the arguments its kernels see.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sgemm {

struct GroupedArgs {
  int M, N, K, groups;
  float alpha, beta;
  const float *A;
  long lda;
  const float *B;
  long ldb, strideB;
  float *C;
  long ldc, strideC;
  const int64_t *offsets;  // device: groups + 1 values
};

// Rows of C by group: C(r, :) = alpha A(r, :) op(B_g) + beta C(r, :).
hipError_t launch_grouped_rows(const GroupedArgs &p, bool tb, int cus, hipStream_t s);

// C_g = alpha A_g^T B_g + beta C_g over the rows (k) of group g.
hipError_t launch_grouped_k(const GroupedArgs &p, int cus, hipStream_t s);

}  // namespace sgemm
