// Activations of the dense layer, their slopes, and vectors of a runtime type.
#pragma once

#include "experts_device.hpp"

namespace mxfp4 {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// 1 / (1 + exp(-v)).  exp overflows to infinity below -88, where the
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

// The lower tail of the normal distribution at -|z|, and exp(-z^2 / 2).
//   Phi(-|z|) = exp(-z^2 / 2) * erfcx(|z| / sqrt 2) / 2
// with erfcx(a) as t * P(t), t = 1 / (1 + 0.4 a): least squares with Lawson's
// weights on [0, 11], relative error 7e-8; past 11 the exponential is 0 in f32.
// In this form the tail keeps its relative precision, which 1 + erf does not.
__device__ __forceinline__ float normal_tail(float z, float &e) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.282842712f * __builtin_fabsf(z));
  e = __expf(-0.5f * z * z);
  float p = 0.04288044f;
  p = p * t - 0.14825743f;
  p = p * t + 0.1004372f;
  p = p * t + 0.06910221f;
  p = p * t + 0.09280704f;
  p = p * t + 0.187831f;
  p = p * t + 0.2033094f;
  p = p * t + 0.22624436f;
  p = p * t + 0.22564584f;
  return 0.5f * e * t * p;
}

// gelu_tanh(z) = z * sigmoid(2 u), u = sqrt(2 / pi) * (z + 0.044715 z^3).  Past
// 30 the sigmoid is 0 or 1, and its cube would overflow first.
constexpr float kTanhC = 1.59576912f, kTanhC3 = 0.0713548163f;  // 2 sqrt(2 / pi), times 0.044715
__device__ __forceinline__ float tanh_clamp(float z) { return __builtin_fminf(__builtin_fmaxf(z, -30.f), 30.f); }

__device__ __forceinline__ float activate(int act, float z) {
  if (act == kActRelu) return z < 0.f ? 0.f : z;
  if (act == kActSilu) return z * sigmoid(z);
  if (act == kActGelu) {
    float e;
    const float tail = normal_tail(z, e);
    return z * (z < 0.f ? tail : 1.0f - tail);
  }
  if (act == kActGeluTanh) {
    const float c = tanh_clamp(z);
    return z * sigmoid(c * (kTanhC + kTanhC3 * c * c));
  }
  return z;
}

// f(z) and f'(z).
__device__ __forceinline__ float activate_slope(int act, float z, float &slope) {
  if (act == kActRelu) {
    slope = z > 0.f ? 1.f : 0.f;
    return z < 0.f ? 0.f : z;
  }
  if (act == kActSilu) {
    const float s = sigmoid(z);
    slope = s + z * s * (1.0f - s);
    return z * s;
  }
  if (act == kActGelu) {
    float e;
    const float tail = normal_tail(z, e);
    const float phi = z < 0.f ? tail : 1.0f - tail;
    slope = phi + 0.398942280f * z * e;
    return z * phi;
  }
  if (act == kActGeluTanh) {
    const float c = tanh_clamp(z);
    const float s = sigmoid(c * (kTanhC + kTanhC3 * c * c));
    slope = s + z * s * (1.0f - s) * (kTanhC + 3.f * kTanhC3 * c * c);
    return z * s;
  }
  slope = 1.f;
  return z;
}

// Four neighbouring elements of an array of a runtime type (MXFP4_TYPE_*), in
// one access where `wide` says that they are aligned to it.
__device__ __forceinline__ v4f load4(const void *p, int type, int64_t i, int wide) {
  v4f v;
  if (type == 2) {
    const float *f = (const float *)p + i;
    if (wide) return *(const v4f *)f;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f[j];
    return v;
  }
  const uint16_t *h = (const uint16_t *)p + i;
  uint16_t d[4];
  if (wide) {
    const u32x2 w = *(const u32x2 *)h;
    d[0] = (uint16_t)w.x, d[1] = (uint16_t)(w.x >> 16), d[2] = (uint16_t)w.y, d[3] = (uint16_t)(w.y >> 16);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = h[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = type == 0 ? __uint_as_float((uint32_t)d[j] << 16) : (float)__builtin_bit_cast(_Float16, d[j]);
  return v;
}

// Two f32 -> two bf16, f16 in one dword, to nearest even.
__device__ __forceinline__ uint32_t f16x2_rne(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

__device__ __forceinline__ void store4(void *p, int type, int64_t i, const v4f &v, int wide) {
  if (type == 2) {
    float *f = (float *)p + i;
    if (wide) {
      *(v4f *)f = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = v[j];
    }
    return;
  }
  const u32x2 d = type == 0 ? u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])}
                            : u32x2{f16x2_rne(v[0], v[1]), f16x2_rne(v[2], v[3])};
  uint16_t *h = (uint16_t *)p + i;
  if (wide) {
    *(u32x2 *)h = d;
  } else {
    h[0] = (uint16_t)d.x, h[1] = (uint16_t)(d.x >> 16), h[2] = (uint16_t)d.y, h[3] = (uint16_t)(d.y >> 16);
  }
}

// Barrier of LDS written by the memory system: the caller has waited for its
// own loads; nothing may move across.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// activate() of eight values, the choice outside.
__device__ __forceinline__ void activate8(int act, float (&z)[8]) {
  switch (act) {
    case kActNone: break;
#define MXFP4_EACH(KIND)                                     \
  case KIND:                                                 \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) z[i] = activate(KIND, z[i]); \
    break;
      MXFP4_EACH(kActRelu)
      MXFP4_EACH(kActSilu)
      MXFP4_EACH(kActGelu)
      MXFP4_EACH(kActGeluTanh)
#undef MXFP4_EACH
  }
}

// Eight neighbouring elements of a runtime type.
__device__ __forceinline__ void load8(const void *p, int type, int64_t i, int wide, float (&v)[8]) {
  const v4f a = load4(p, type, i, wide), b = load4(p, type, i + 4, wide);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
}

__device__ __forceinline__ void unpack8(const u32x4 &d, int type, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = d[j];
    if (type == 0) {
      v[2 * j] = __uint_as_float(w << 16);
      v[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
    } else {
      const f16x2 h = __builtin_bit_cast(f16x2, w);
      v[2 * j] = (float)h.x;
      v[2 * j + 1] = (float)h.y;
    }
  }
}

// Cache policy of a store: past the caches.  What a large product writes would
// displace what it reads from L2 otherwise (8192 x 16384 x 2048, bf16: 232 us
// through the caches, 193 past them).
constexpr int kPastCaches = 2;

// ... at a byte offset of a buffer, where an offset out of range reads zeros and
// stores nothing.  `wide`: 16 bytes at a time.
struct Raw8 {
  u32x4 d[2];  // the second of f32 only
};
__device__ __forceinline__ Raw8 load_raw8(const __amdgpu_buffer_rsrc_t &r, int type, int off, int wide) {
  Raw8 v;
  if (wide) {
    v.d[0] = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    if (type == 2) v.d[1] = __builtin_amdgcn_raw_buffer_load_b128(r, off, 16, 0);
  } else if (type == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.d[i >> 2][i & 3] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 4 * i, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.d[0][i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 4 * i, 0) |
                  (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 4 * i + 2, 0) << 16;
  }
  return v;
}
__device__ __forceinline__ void add_raw8(const Raw8 &r, int type, float (&v)[8]) {
  if (type == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(r.d[i >> 2][i & 3]);
  } else {
    float f[8];
    unpack8(r.d[0], type, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += f[i];
  }
}
__device__ __forceinline__ void store8(const __amdgpu_buffer_rsrc_t &r, int type, int off, const float (&v)[8], int wide) {
  if (type == 2) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      u32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = __float_as_uint(v[j + i]);
      if (wide) {
        __builtin_amdgcn_raw_buffer_store_b128(d, r, off, 4 * j, kPastCaches);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) __builtin_amdgcn_raw_buffer_store_b32(d[i], r, off, 4 * (j + i), 0);
      }
    }
    return;
  }
  u32x4 d;
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = type == 0 ? bf16x2_rne(v[2 * j], v[2 * j + 1]) : f16x2_rne(v[2 * j], v[2 * j + 1]);
  if (wide) {
    __builtin_amdgcn_raw_buffer_store_b128(d, r, off, 0, kPastCaches);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)d[i], r, off, 4 * i, 0);
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(d[i] >> 16), r, off, 4 * i + 2, 0);
    }
  }
}

}  // namespace mxfp4
