// C ABI of the expert operators: argument checks and launches.  Every check
// runs on the host before anything is enqueued.
#include "../../include/mxfp4.h"
#include "experts_internal.hpp"
#include "mxfp4_internal.hpp"

using namespace mxfp4;

namespace {

const int64_t kMaxBytes = (int64_t)1 << 31;  // 32-bit offsets inside the kernels
const int64_t kMaxRows = (int64_t)1 << 20;
const int64_t kMaxGroups = 4096;

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

// The caller's workspace if it gave one, else the library's, behind the
// ticket words that the split-K products keep at zero; `held` keeps that one
// for this call while it lives.
mxfp4_status_t take_workspace(void *given, size_t given_bytes, size_t need, hipStream_t stream, HeldWorkspace *held,
                              void **out) {
  *out = given;
  if (given) return given_bytes >= need && aligned(given, 256) ? MXFP4_OK : MXFP4_ERR_WORKSPACE;
  if (need == 0) return MXFP4_OK;
  const mxfp4_status_t st = hold_workspace(kTicketBytes + need, stream, held);
  if (st == MXFP4_OK) *out = (char *)held->ptr + kTicketBytes;
  return st;
}

}  // namespace

extern "C" {

mxfp4_status_t mxfp4_reserve_bytes(size_t bytes, mxfp4_stream_t stream) {
  if (bytes > ((size_t)1 << 46)) return MXFP4_ERR_UNSUPPORTED;
  return ready_workspace(bytes ? kTicketBytes + bytes : 0, (hipStream_t)stream);
}

size_t mxfp4_moe_route_workspace_bytes(int64_t T, int64_t E) {
  return T < 1 || E < 1 || T > kMaxRows || E > kRouteMaxExperts ? 0 : route_workspace_bytes(T, E);
}

mxfp4_status_t mxfp4_moe_route(const void *logits, int x_type, int64_t ld, const float *bias, int64_t T, int64_t E,
                               int64_t k, int score, int renormalize, int32_t *ids, float *weights,
                               int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace, size_t workspace_bytes,
                               mxfp4_stream_t stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || ld < E || !known_type(x_type) || !offsets) return MXFP4_ERR_INVALID_ARG;
  if (score != MXFP4_SCORE_SOFTMAX && score != MXFP4_SCORE_SIGMOID) return MXFP4_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !ids || !weights || !rows || !pos)) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(logits, size_of(x_type)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4))
    return MXFP4_ERR_INVALID_ARG;
  if (T > kMaxRows || E > kRouteMaxExperts || k > kRouteMaxChoices || ld > ((int64_t)1 << 40))
    return MXFP4_ERR_UNSUPPORTED;
  HeldWorkspace held;
  void *ws = nullptr;
  const mxfp4_status_t st =
      take_workspace(workspace, workspace_bytes, route_workspace_bytes(T, E), (hipStream_t)stream, &held, &ws);
  if (st != MXFP4_OK) return st;
  RouteArgs a{};
  a.logits = logits;
  a.x_type = x_type;
  a.ld = ld;
  a.bias = bias;
  a.T = (int)T;
  a.E = (int)E;
  a.k = (int)k;
  a.score = score;
  a.renorm = renormalize != 0;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.rows = rows;
  a.pos = pos;
  a.hist = (uint16_t *)ws;
  return hip_status(launch_route(a, (hipStream_t)stream));
}

size_t mxfp4_gemm_grouped_workspace_bytes(int64_t R, int64_t K, int64_t experts) {
  if (R < 1 || K < 1 || experts < 1 || R > kMaxRows || K > ((int64_t)1 << 17) || experts > kMaxGroups) return 0;
  return grouped_workspace_bytes(R, K, experts);
}

mxfp4_status_t mxfp4_gemm_grouped(const void *A, int64_t lda, int64_t a_rows, const void *Bq_sh, const void *Bs_sh,
                                  int64_t experts, const int32_t *offsets, const int32_t *rows, int64_t repeat,
                                  void *C, int64_t ldc, int64_t R, int64_t N, int64_t K, int gated, void *workspace,
                                  size_t workspace_bytes, mxfp4_stream_t stream) {
  if (R < 0 || a_rows < 0 || N < 1 || K < 1 || experts < 1 || repeat < 1) return MXFP4_ERR_INVALID_ARG;
  if (!Bq_sh || !Bs_sh || !offsets || (R > 0 && !C) || (a_rows > 0 && !A)) return MXFP4_ERR_INVALID_ARG;
  if (lda < K || ldc < (gated ? N / 2 : N)) return MXFP4_ERR_INVALID_ARG;
  if (K % 32 != 0 || N % 16 != 0 || (gated && N % 32 != 0)) return MXFP4_ERR_UNSUPPORTED;
  if (R > kMaxRows || a_rows > kMaxRows || experts > kMaxGroups || repeat > INT32_MAX || !matrix_fits(N, K) ||
      N > kMaxRows || K > ((int64_t)1 << 17) || lda > ((int64_t)1 << 30) || ldc > ((int64_t)1 << 22))
    return MXFP4_ERR_UNSUPPORTED;
  if (!aligned(A, 16) || lda % 8 != 0 || !aligned(Bq_sh, 16) || !aligned(Bs_sh, 16) || !aligned(offsets, 4) ||
      !aligned(rows, 4) || !aligned(C, 2))
    return MXFP4_ERR_INVALID_ARG;
  if (R == 0) return MXFP4_OK;
  HeldWorkspace held;
  void *ws = nullptr;
  const mxfp4_status_t st = take_workspace(workspace, workspace_bytes, grouped_workspace_bytes(R, K, experts),
                                           (hipStream_t)stream, &held, &ws);
  if (st != MXFP4_OK) return st;
  GroupedArgs a{};
  a.A = (const uint16_t *)A;
  a.lda = lda;
  a.a_rows = a_rows;
  a.Bw = (const uint8_t *)Bq_sh;
  a.Bs = (const uint8_t *)Bs_sh;
  a.offsets = offsets;
  a.rows = rows;
  a.C = (uint16_t *)C;
  a.ldc = ldc;
  a.R = (int)R;
  a.N = (int)N;
  a.K = (int)K;
  a.E = (int)experts;
  a.repeat = (int)repeat;
  a.gated = gated != 0;
  a.sw = sw_quant();
  a.ws = (uint8_t *)ws;
  return hip_status(launch_grouped(a, (hipStream_t)stream));
}

mxfp4_status_t mxfp4_moe_combine(const void *y, int y_type, int64_t ld_y, int64_t rows, const float *weights,
                                 const int32_t *pos, const void *residual, int64_t ld_res, void *out, int out_type,
                                 int64_t ld_out, int64_t T, int64_t k, int64_t N, mxfp4_stream_t stream) {
  if (T < 0 || rows < 0 || N < 1 || k < 1 || !known_type(y_type) || !known_type(out_type)) return MXFP4_ERR_INVALID_ARG;
  if (ld_y < N || ld_out < N || (residual && ld_res < N)) return MXFP4_ERR_INVALID_ARG;
  if (T > 0 && (!weights || !out || (rows > 0 && !y))) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(y, size_of(y_type)) || !aligned(weights, 4) || !aligned(pos, 4) ||
      !aligned(residual, size_of(out_type)) || !aligned(out, size_of(out_type)))
    return MXFP4_ERR_INVALID_ARG;
  const int64_t far = (int64_t)1 << 40;  // row counts and strides whose products stay below 2^63 bytes
  if (N >= INT32_MAX - 4096 || k > kMaxRows || T > ((int64_t)1 << 20) * 64 || rows > ((int64_t)1 << 30) ||
      ld_y > far / 1024 || ld_out > far / 1024 || (residual && ld_res > far / 1024))
    return MXFP4_ERR_UNSUPPORTED;
  if (T == 0) return MXFP4_OK;
  CombineArgs a{y,        y_type, ld_y,     rows,   weights, pos, residual,
                ld_res,   out,    out_type, ld_out, T,       N,   (int)k};
  return hip_status(launch_combine(a, (hipStream_t)stream));
}

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
