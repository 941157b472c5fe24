// Host-side declarations of the dense layer and its gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxfp4 {

// Rows of bf16 quantized into the layout of a prepared matrix [rows, K]: codes
// of 16-row group g, 32-element group t at (g * (K / 32) + t) * 256, and
// shuffled scales.  Rows past the last one of their 16-row group are zeros.
inline size_t packed_codes_bytes(int64_t rows, int64_t K) { return (size_t)((rows + 15) / 16) * (size_t)K * 8; }
inline size_t packed_scale_bytes(int64_t rows, int64_t K) {
  return (size_t)((rows + 255) / 256 * 256) * (size_t)((K / 32 + 7) / 8 * 8);
}
inline size_t packed_bytes(int64_t rows, int64_t K) {
  return (packed_codes_bytes(rows, K) + 255) / 256 * 256 + packed_scale_bytes(rows, K);
}

struct LinearArgs {
  const uint16_t *x;
  int64_t ldx;
  const uint8_t *Bw, *Bs;
  const void *bias;  // or null
  int bias_type, act, gated;
  const void *residual;  // or null; of y's type
  int64_t ld_res;
  void *y;
  int y_type;
  int64_t ldy;
  uint16_t *pre;  // or null
  int64_t ld_pre;
  int M, N, K, sw;
  uint8_t *ws;
  // set by launch_linear
  uint8_t *codes, *scales;  // of the quantized rows, in ws
  int wide_y, wide_pre, wide_bias;  // whether four columns go in one access (y's also of the residual)
  int line_y, line_pre;             // ... or 16 bytes
};

size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear(LinearArgs a, hipStream_t stream);
hipError_t launch_linear_tile(const LinearArgs &a, hipStream_t stream);  // rows quantized

struct GradPreArgs {
  const void *dy;
  int dy_type;
  int64_t ld_dy;
  const uint16_t *pre;  // or null where the activation is none
  int64_t ld_pre;
  int act, gated;
  uint16_t *dz;
  int64_t ld_dz;
  float *dbias;  // or null
  int M, N;
  float *partial;  // [chunks][N] in the workspace
  int chunks, chunk_rows;
  int wide;
};

size_t grad_pre_workspace_bytes(int64_t M, int64_t N);
hipError_t launch_grad_pre(GradPreArgs a, hipStream_t stream);

// out[i, k] = sum_j P[i, j] * T[j, k] with T an MXFP4 matrix in prepared form.
struct GradProductArgs {
  const uint16_t *P;  // [I, J] rows, or (transposed) [J, I] rows
  int64_t ldp;
  int transposed;
  const uint8_t *codes, *scales;  // of T [J, K]
  void *out;
  int out_type;
  int64_t ld_out;
  int I, J, K;
  float *partial;  // [splits][I][K] in the workspace, if splits > 1
  int splits, split_stages;
  int wide, wide4;  // whether out takes 16 bytes, or four elements, in one access
};

size_t grad_product_workspace_bytes(int64_t I, int64_t J, int64_t K, bool transposed);
hipError_t launch_grad_product(GradProductArgs a, hipStream_t stream);

// Quantize `rows` rows of bf16, ld elements apart, into the prepared layout.
hipError_t launch_pack_rows(const uint16_t *x, int64_t ld, int64_t rows, int64_t K, uint8_t *codes, uint8_t *scales,
                            bool sw, hipStream_t stream);

}  // namespace mxfp4
