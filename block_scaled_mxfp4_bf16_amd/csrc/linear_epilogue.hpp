// What the dense layer does with its sums.
#pragma once

#include "linear_device.hpp"
#include "linear_internal.hpp"

namespace mxfp4 {

__device__ __forceinline__ v4f mfma_fp4(const u32x4 &a, const u32x4 &b, const v4f &c, uint32_t sa, uint32_t sb) {
  const v8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Output columns col .. col + 3 of one row from their f32 sums (gated: of the
// gate's columns in z and of the up projection's in up).  Everything is f32
// until y and the kept z are rounded, once each; the activation takes the
// unrounded z.
__device__ __forceinline__ void linear_emit(const LinearArgs &a, int row, int col, v4f z, v4f up) {
  const int half = a.N >> 1;
  if (a.bias) {
    z += load4(a.bias, a.bias_type, col, 0);
    if (a.gated) up += load4(a.bias, a.bias_type, half + col, 0);
  }
  if (a.pre) {
    store4(a.pre, 0, (int64_t)row * a.ld_pre + col, z, a.wide_pre);
    if (a.gated) store4(a.pre, 0, (int64_t)row * a.ld_pre + half + col, up, a.wide_pre);
  }
  v4f y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = activate(a.act, z[i]);
  if (a.gated) y *= up;
  if (a.residual) y += load4(a.residual, a.y_type, (int64_t)row * a.ld_res + col, a.wide_y);
  store4(a.y, a.y_type, (int64_t)row * a.ldy + col, y, a.wide_y);
}

}  // namespace mxfp4
