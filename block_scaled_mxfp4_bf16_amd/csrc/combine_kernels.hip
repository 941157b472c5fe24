// The weighted sum of a token's expert rows:
//   out[t, n] = residual[t, n] + sum_j w[t, j] * y[pos[t, j], n]
// in f32, the choices in order and the residual last, rounded once.
//
// Reading y bounds it.  A thread takes 16 bytes (8 columns) of a token; the
// loads of all choices (in runs of kAhead) go out before the first is used,
// so a token pays the memory latency once, not once per choice.
#include "experts_device.hpp"
#include "experts_internal.hpp"

namespace mxfp4 {

namespace {

constexpr int kAhead = 8;  // choices whose loads are in flight together

// C consecutive elements of an array of type YT as they are loaded.
template <class YT, int C>
struct Piece {
  YT v[C];
};

template <class YT, int C>
__device__ __forceinline__ Piece<YT, C> load_piece(const YT *p) {
  Piece<YT, C> r;
  if constexpr (C == 1) {
    r.v[0] = *p;
  } else {
    union {
      u32x4 u[C * sizeof(YT) / 16];
      Piece<YT, C> p;
    } b;
#pragma unroll
    for (int i = 0; i < (int)(C * sizeof(YT) / 16); ++i) b.u[i] = ((const u32x4 *)p)[i];
    r = b.p;
  }
  return r;
}

}  // namespace

// Thread: columns [C * x, C * x + C) of token blockIdx.y (+ gridDim.y ...).
template <class YT, class OT, int C>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a) {
  const int64_t n = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * C;
  if (n >= a.N) return;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    Piece<OT, C> res;
    if (a.residual) res = load_piece<OT, C>((const OT *)a.residual + t * a.ld_res + n);
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
      Piece<YT, C> y[kAhead];
      float w[kAhead];
      bool live[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i;
        int64_t row = -1;
        if (j < a.k) row = a.pos ? (int64_t)a.pos[t * a.k + j] : t * a.k + j;
        live[i] = row >= 0 && row < a.rows;
        w[i] = live[i] ? a.weights[t * a.k + j] : 0.f;
        if (live[i]) y[i] = load_piece<YT, C>((const YT *)a.y + row * a.ld_y + n);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (live[i])
#pragma unroll
          for (int c = 0; c < C; ++c) acc[c] += w[i] * (float)y[i].v[c];
    }
    if (a.residual)
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += (float)res.v[c];
    OT *out = (OT *)a.out + t * a.ld_out + n;
    if constexpr (C == 1) {
      *out = (OT)acc[0];
    } else {
      union {
        u32x4 u[C * sizeof(OT) / 16];
        OT v[C];
      } b;
#pragma unroll
      for (int c = 0; c < C; ++c) b.v[c] = (OT)acc[c];
#pragma unroll
      for (int i = 0; i < (int)(C * sizeof(OT) / 16); ++i) ((u32x4 *)out)[i] = b.u[i];
    }
  }
}

template <class YT, class OT>
static hipError_t run_combine(const CombineArgs &a, hipStream_t stream) {
  const auto vector_rows = [&](const void *p, int64_t ld, size_t size) {
    return ((uintptr_t)p & 15) == 0 && ld * (int64_t)size % 16 == 0;
  };
  const unsigned ty = (unsigned)(a.T < 65535 ? a.T : 65535);
  if (a.N % 8 == 0 && vector_rows(a.y, a.ld_y, sizeof(YT)) && vector_rows(a.out, a.ld_out, sizeof(OT)) &&
      (!a.residual || vector_rows(a.residual, a.ld_res, sizeof(OT)))) {
    const int threads = a.N >= 2048 ? 256 : 64;
    combine_kernel<YT, OT, 8><<<dim3((unsigned)((a.N / 8 + threads - 1) / threads), ty), threads, 0, stream>>>(a);
  } else {
    combine_kernel<YT, OT, 1><<<dim3((unsigned)((a.N + 255) / 256), ty), 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <class YT>
static hipError_t run_combine_from(const CombineArgs &a, hipStream_t stream) {
  if (a.out_type == MXFP4_TYPE_BF16) return run_combine<YT, __bf16>(a, stream);
  if (a.out_type == MXFP4_TYPE_F16) return run_combine<YT, _Float16>(a, stream);
  return run_combine<YT, float>(a, stream);
}

hipError_t launch_combine(const CombineArgs &a, hipStream_t stream) {
  if (a.y_type == MXFP4_TYPE_BF16) return run_combine_from<__bf16>(a, stream);
  if (a.y_type == MXFP4_TYPE_F16) return run_combine_from<_Float16>(a, stream);
  return run_combine_from<float>(a, stream);
}

}  // namespace mxfp4
