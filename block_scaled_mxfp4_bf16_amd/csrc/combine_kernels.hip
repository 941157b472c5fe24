// The weighted sum of a token's expert rows:
//   out[t, n] = residual[t, n] + sum_j w[t, j] * y[pos[t, j], n]
// in f32, the choices in order and the residual last, rounded once.
//
// Reading y bounds it.  A thread takes 16 bytes (8 columns) of a token; the
// loads of all choices (in runs of kAhead) go out before the first is used,
// so a token pays the memory latency once, not once per choice.  Measured: 8
// rows of 2048 for 4096 tokens 28.6 us, 5.9 TB/s; 8 rows of 7168 for 4 tokens 4.4
// us, two dependent loads behind a launch.
#include "experts_device.hpp"
#include "experts_internal.hpp"

namespace mxfp4 {

namespace {

constexpr int kAhead = 8;  // choices whose loads are in flight together

// The choices' places and weights are the same for all lanes and not written
// here: read through the scalar cache, all at once.  As vector loads, each
// waited for before its row's own load, 8 choices of 4096 tokens of 2048 columns took
// 40.8 us instead of 35.8.
template <class T>
__device__ __forceinline__ const __attribute__((address_space(4))) T *uniform(const T *p) {
  return (const __attribute__((address_space(4))) T *)p;
}

// C consecutive elements of an array of type YT as they are loaded.
template <class YT, int C>
struct Piece {
  YT v[C];
};

template <class YT, int C, bool ONCE>
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
    for (int i = 0; i < (int)(C * sizeof(YT) / 16); ++i) b.u[i] = ONCE ? __builtin_nontemporal_load((const u32x4 *)p + i) : ((const u32x4 *)p)[i];
    r = b.p;
  }
  return r;
}

}  // namespace

// ONCE: the rows are too many to be found in a cache again, and neither they
// nor the sums are kept there.
// Thread: columns [C * x, C * x + C) of token blockIdx.y (+ gridDim.y ...).
template <class YT, class OT, int C, bool ONCE>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a) {
  const int64_t n = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * C;
  if (n >= a.N) return;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    Piece<OT, C> res;
    if (a.residual) res = load_piece<OT, C, ONCE>((const OT *)a.residual + t * a.ld_res + n);
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
      Piece<YT, C> y[kAhead];
      float w[kAhead];
      bool live[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i;
        int64_t row = -1;
        w[i] = 0.f;
        if (j < a.k) {
          row = a.pos ? (int64_t)uniform(a.pos)[t * a.k + j] : t * a.k + j;
          w[i] = uniform(a.weights)[t * a.k + j];
        }
        live[i] = row >= 0 && row < a.rows;
        if (live[i]) y[i] = load_piece<YT, C, ONCE>((const YT *)a.y + row * a.ld_y + n);
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
      for (int i = 0; i < (int)(C * sizeof(OT) / 16); ++i) {
        if constexpr (ONCE)
          __builtin_nontemporal_store(b.u[i], (u32x4 *)out + i);
        else
          ((u32x4 *)out)[i] = b.u[i];
      }
    }
  }
}

// Bytes of y from which on they are read past the caches.  8 rows of 2048 a
// token, both ways: 67 MB 14.4 and 15.0 us; 134 MB 35.9 and 28.9 cold, 29.0
// and 27.9 just written by the product; 268 MB 67.7 and 56.0.
constexpr int64_t kOnceBytes = (int64_t)96 << 20;

template <class YT, class OT>
static hipError_t run_combine(const CombineArgs &a, hipStream_t stream) {
  const auto vector_rows = [&](const void *p, int64_t ld, size_t size) {
    return ((uintptr_t)p & 15) == 0 && ld * (int64_t)size % 16 == 0;
  };
  const unsigned ty = (unsigned)(a.T < 65535 ? a.T : 65535);
  if (a.N % 8 == 0 && vector_rows(a.y, a.ld_y, sizeof(YT)) && vector_rows(a.out, a.ld_out, sizeof(OT)) &&
      (!a.residual || vector_rows(a.residual, a.ld_res, sizeof(OT)))) {
    const int threads = a.N >= 2048 ? 256 : 64;
    const dim3 grid((unsigned)((a.N / 8 + threads - 1) / threads), ty);
    // compared by division: the product of the three could overflow
    if (a.T >= kOnceBytes / (int64_t)sizeof(YT) / a.N / a.k)
      combine_kernel<YT, OT, 8, true><<<grid, threads, 0, stream>>>(a);
    else
      combine_kernel<YT, OT, 8, false><<<grid, threads, 0, stream>>>(a);
  } else {
    combine_kernel<YT, OT, 1, false><<<dim3((unsigned)((a.N + 255) / 256), ty), 256, 0, stream>>>(a);
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
