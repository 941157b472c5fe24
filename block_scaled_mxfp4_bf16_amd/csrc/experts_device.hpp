// Device helpers of the expert operators.
#pragma once

#include "mxfp4_device.hpp"

namespace mxfp4 {

template <int V>
constexpr int kLog2 = V <= 1 ? 0 : 1 + kLog2<V / 2>;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// Swap the upper 32 lanes of a with the lower 32 of b.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
  const u32x2 r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r.x;
  b = r.y;
}
// Swap lanes 16-31 of a with lanes 0-15 of b, and 48-63 with 32-47.
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
  const u32x2 r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r.x;
  b = r.y;
}

// Between LDS accesses of different lanes of one wave to the same place: the
// hardware does a wave's accesses in order, so this only keeps the compiler
// from moving one past the other, which a lane's own addresses would allow.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// silu(g) * u.  exp(-g) overflows to infinity for g below -88, where the
// quotient is the right -0.  The reciprocal is the hardware's, within 1 ulp:
// next to the exponential's own error it costs nothing, and a divide takes ten
// instructions more.
__device__ __forceinline__ float gated_silu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

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
