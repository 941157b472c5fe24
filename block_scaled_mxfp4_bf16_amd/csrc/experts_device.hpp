// Device helpers of the expert operators.
#pragma once

#include "mxfp4_device.hpp"

namespace mxfp4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// silu(g) * u.  exp(-g) overflows to infinity for g below -88, where the
// quotient is the right -0.
__device__ __forceinline__ float gated_silu(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// Element `i` of an array of the given type (MXFP4_TYPE_*), rounded to
// nearest even, written through vector stores.
__device__ __forceinline__ void store_as(void *p, int type, size_t i, float v) {
  if (type == 0)
    ((__bf16 *)p)[i] = (__bf16)v;
  else if (type == 1)
    ((_Float16 *)p)[i] = (_Float16)v;
  else
    ((float *)p)[i] = v;
}

}  // namespace mxfp4
