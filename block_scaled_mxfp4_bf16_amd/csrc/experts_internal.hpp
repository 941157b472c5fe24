// Host-side declarations of the expert operators: the row product with
// unquantized activations, the router, the grouped product and the sum of a
// token's expert rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

}  // namespace mxfp4
