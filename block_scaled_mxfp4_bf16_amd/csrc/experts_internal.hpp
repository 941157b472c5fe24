// Host-side declarations of the expert operators: the row product with
// unquantized activations, the router, the grouped product and the sum of a
// token's expert rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mxfp4.h"

namespace mxfp4 {

struct GemvArgs {
  const void *x;
  int x_type;
  int64_t ldx;
  const uint8_t *Bw, *Bs;
  const int32_t *ids;  // one matrix per row, or null
  int experts;
  void *y;
  int y_type;
  int64_t ldy;
  int M, N, K, repeat, gated;
};

hipError_t launch_gemv(const GemvArgs &a, hipStream_t stream);

// Largest number of experts and of choices of the router.
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxChoices = 32;

struct RouteArgs {
  const void *logits;
  int x_type;
  int64_t ld;
  const float *bias;  // or null
  int T, E, k, score, renorm;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *rows, *pos;
  uint16_t *hist;  // [E][2^hist_shift] counts of each block, unless T is small
  int blocks, per_block, hist_shift;
};

size_t route_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);

struct GroupedArgs {
  const uint16_t *A;
  int64_t lda, a_rows;
  const uint8_t *Bw, *Bs;
  const int32_t *offsets;
  const int32_t *rows;  // or null: output row p takes row p of A
  uint16_t *C;
  int64_t ldc;
  int R, N, K, E, repeat, gated, sw;
  uint8_t *ws;
  // set by launch_grouped: in ws, the list of units and the packed rows
  int4 *plan;
  uint8_t *codes, *scales;
  int quads, max_units, unit_rows, unit_shift;
  int pairs;  // the order of the packed rows' scales
};

size_t grouped_workspace_bytes(int64_t R, int64_t K, int64_t E);
hipError_t launch_grouped(GroupedArgs a, hipStream_t stream);

struct CombineArgs {
  const void *y;
  int y_type;
  int64_t ld_y, rows;
  const float *weights;
  const int32_t *pos;    // or null: row t * k + j
  const void *residual;  // or null; of the output's type
  int64_t ld_res;
  void *out;
  int out_type;
  int64_t ld_out;
  int64_t T, N;
  int k;
};

hipError_t launch_combine(const CombineArgs &a, hipStream_t stream);

}  // namespace mxfp4
