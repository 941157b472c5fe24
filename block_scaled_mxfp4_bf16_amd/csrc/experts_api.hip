// C ABI of the expert operators: argument checks and launches.  Every check
// runs on the host before anything is enqueued.
#include "../../include/mxfp4.h"
#include "experts_internal.hpp"
#include "mxfp4_internal.hpp"

using namespace mxfp4;

namespace {

const int64_t kMaxBytes = (int64_t)1 << 31;  // 32-bit offsets inside the kernels
const int64_t kMaxRows = (int64_t)1 << 20;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int64_t pad_to(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline bool known_type(int t) { return t == MXFP4_TYPE_BF16 || t == MXFP4_TYPE_F16 || t == MXFP4_TYPE_F32; }

inline int64_t size_of(int t) { return t == MXFP4_TYPE_F32 ? 4 : 2; }

// Whether 32-bit offsets reach all of one prepared matrix; sizes are
// compared by division, so that no product overflows.
inline bool matrix_fits(int64_t N, int64_t K) {
  if (N >= kMaxBytes || K >= kMaxBytes) return false;
  return N <= (kMaxBytes - 1) / ((K + 1) / 2) && pad_to(N, 256) <= (kMaxBytes - 1) / pad_to(K / 32 + 1, 8);
}

}  // namespace

extern "C" {

mxfp4_status_t mxfp4_gemv(const void *x, int x_type, int64_t ldx, const void *Bq_sh, const void *Bs_sh,
                          const int32_t *ids, int64_t experts, void *y, int y_type, int64_t ldy, int64_t M, int64_t N,
                          int64_t K, int64_t repeat, int gated, mxfp4_stream_t stream) {
  if (!x || !Bq_sh || !Bs_sh || !y || !known_type(x_type) || !known_type(y_type)) return MXFP4_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 1 || experts < 1 || repeat < 1 || (!ids && repeat != 1)) return MXFP4_ERR_INVALID_ARG;
  if (ldx < K || ldy < (gated ? N / 2 : N)) return MXFP4_ERR_INVALID_ARG;
  if (K % 32 != 0 || N % 16 != 0 || (gated && N % 32 != 0)) return MXFP4_ERR_UNSUPPORTED;
  if (M > kMaxRows || experts > INT32_MAX || repeat > INT32_MAX || !matrix_fits(N, K)) return MXFP4_ERR_UNSUPPORTED;
  if (ldx > (kMaxBytes - 1) / (64 * size_of(x_type))) return MXFP4_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || ldx * size_of(x_type) % 16 != 0 || !aligned(Bq_sh, 16) || !aligned(Bs_sh, 16) ||
      !aligned(ids, 4) || !aligned(y, size_of(y_type)))
    return MXFP4_ERR_INVALID_ARG;
  GemvArgs a{x,      x_type, ldx,    (const uint8_t *)Bq_sh, (const uint8_t *)Bs_sh, ids,        (int)experts, y,
             y_type, ldy,    (int)M, (int)N,                 (int)K,                 (int)repeat, gated != 0};
  return hip_status(launch_gemv(a, (hipStream_t)stream));
}

}  // extern "C"
