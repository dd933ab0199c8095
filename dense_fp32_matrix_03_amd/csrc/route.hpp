// route.hpp -- routing of tokens to experts and the movement of their rows
// (include/sgemm_route.h): arguments of the kernels and host-side launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace sgemm {

struct RouteArgs {
  int tokens, experts, topk;
  bool sigmoid, renormalize;
  const void *logits;
  long ldl;
  const float *bias;
  int groups, keep, group_top;
  float scale;
  int32_t *picks;
  float *weights;
  FastDiv by_size;  // experts of a group
  int group_share;  // lanes of a group: a power of two, groups * group_share <= 64
};
hipError_t launch_route(const RouteArgs &p, bool bf16, hipStream_t s);

struct RouteBackArgs {
  int tokens, experts, topk;
  bool sigmoid, renormalize;
  const void *logits;
  long ldl;
  float scale;
  const int32_t *picks;
  const float *dweights;
  void *dlogits;
  long ldd;
};
hipError_t launch_route_backward(const RouteBackArgs &p, bool bf16, hipStream_t s);

// Pairs are counted in chunks of consecutive ones, a work-group each.
struct PlanArgs {
  int pairs, first, groups;
  int chunk, chunks;
  const int32_t *picks;
  int64_t *offsets;
  int32_t *sources, *places;
  int *counts;  // [chunks][groups], in the workspace
};
constexpr int kPlanChunk = 2048;  // pairs of a chunk, at least where there are several
constexpr int kPlanChunks = 256;  // chunks, at most
inline int plan_chunk(long pairs) {  // a multiple of 256
  const long share = (pairs + kPlanChunks - 1) / kPlanChunks;
  const long least = pairs < kPlanChunk ? pairs : kPlanChunk;
  const long chunk = share > least ? share : least;
  return (int)((chunk < 1 ? 1 : chunk) + 255) / 256 * 256;
}
inline int plan_chunks(long pairs) { return (int)((pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs)); }
hipError_t launch_route_plan(const PlanArgs &p, hipStream_t s);

// Columns of a row that a wave moves, in bytes of the row.
constexpr int kRowPiece = 4096;
struct RowsArgs {
  int rows, topk, N;      // rows: those that are written (tokens of a combination)
  int limit;              // indices below it are in range
  const void *X;
  long ldx;
  const int32_t *index;   // sources, or places
  const float *weights;
  void *Y;
  long ldy;
  FastDiv by_pieces;      // pieces of a row
  int pieces;
};
hipError_t launch_rows_gather(const RowsArgs &p, bool bf16, hipStream_t s);
hipError_t launch_rows_combine(const RowsArgs &p, bool bf16, hipStream_t s);

struct RowsBackArgs {
  int pairs, topk, N, rows;
  const void *X;
  long ldx;
  const void *dY;
  long lddy;
  const int32_t *places;
  const float *weights;
  void *dX;
  long lddx;
  float *dweights;
};
hipError_t launch_rows_combine_backward(const RowsBackArgs &p, bool bf16, hipStream_t s);

}  // namespace sgemm
