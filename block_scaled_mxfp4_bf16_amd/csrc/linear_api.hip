// C ABI of the dense layer and its gradients: argument checks and launches.
// Every check runs on the host before anything is enqueued.
#include "api_checks.hpp"
#include "linear_internal.hpp"

using namespace mxfp4;

namespace {

const int64_t kMaxK = (int64_t)1 << 17;
const int64_t kMaxStride = (int64_t)1 << 20;  // of any row, in elements

inline bool known_act(int act) { return act >= MXFP4_ACT_NONE && act <= MXFP4_ACT_GELU_TANH; }

// Sizes and the prepared matrix [N, K] that all but the activation's gradient share.
inline bool sizes_fit(int64_t M, int64_t N, int64_t K) {
  return K % 32 == 0 && N % 16 == 0 && M <= kMaxRows && N <= kMaxRows && K <= kMaxK;
}

// Whether vectors of four elements of `size` bytes at p, rows ld apart, are aligned.
inline bool wide4(const void *p, int64_t ld, int64_t size) { return !p || (aligned(p, 4 * size) && ld % 4 == 0); }

// ... and pieces of 16 bytes.
inline bool lines(const void *p, int64_t ld, int64_t size) { return !p || (aligned(p, 16) && ld * size % 16 == 0); }

// A matrix that the kernels read in 16-byte pieces of bf16.
inline bool vector_rows(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

extern "C" {

size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M < 1 || N < 1 || K < 1 || !sizes_fit(M, N, K) ? 0 : linear_workspace_bytes(M, N, K);
}

mxfp4_status_t mxfp4_linear(const void *x, int64_t ldx, const void *Bq_sh, const void *Bs_sh, const void *bias,
                            int bias_type, int activation, int gated, const void *residual, int64_t ld_res, void *y,
                            int y_type, int64_t ldy, void *pre, int64_t ld_pre, int64_t M, int64_t N, int64_t K,
                            void *workspace, size_t workspace_bytes, mxfp4_stream_t stream) {
  const int64_t cols = gated ? N / 2 : N;
  if (M < 0 || N < 1 || K < 1 || !known_act(activation) || !known_type(y_type) || (bias && !known_type(bias_type)))
    return MXFP4_ERR_INVALID_ARG;
  if (!Bq_sh || !Bs_sh || (M > 0 && (!x || !y))) return MXFP4_ERR_INVALID_ARG;
  if (ldx < K || ldy < cols || (residual && ld_res < cols) || (pre && ld_pre < N)) return MXFP4_ERR_INVALID_ARG;
  if (!sizes_fit(M, N, K) || (gated && N % 32 != 0) || !matrix_fits(N, K) || ldx > kMaxStride || ldy > kMaxStride ||
      (residual && ld_res > kMaxStride) || (pre && ld_pre > kMaxStride))
    return MXFP4_ERR_UNSUPPORTED;
  if (!vector_rows(x, ldx) || !aligned(Bq_sh, 16) || !aligned(Bs_sh, 16) || (bias && !aligned(bias, size_of(bias_type))) ||
      !aligned(residual, size_of(y_type)) || !aligned(y, size_of(y_type)) || !aligned(pre, 2))
    return MXFP4_ERR_INVALID_ARG;
  if (M == 0) return MXFP4_OK;
  HeldWorkspace held;
  void *ws = nullptr;
  const mxfp4_status_t st =
      take_workspace(workspace, workspace_bytes, linear_workspace_bytes(M, N, K), (hipStream_t)stream, &held, &ws);
  if (st != MXFP4_OK) return st;
  LinearArgs a{};
  a.x = (const uint16_t *)x;
  a.ldx = ldx;
  a.Bw = (const uint8_t *)Bq_sh;
  a.Bs = (const uint8_t *)Bs_sh;
  a.bias = bias;
  a.bias_type = bias_type;
  a.act = activation;
  a.gated = gated != 0;
  a.residual = residual;
  a.ld_res = ld_res;
  a.y = y;
  a.y_type = y_type;
  a.ldy = ldy;
  a.pre = (uint16_t *)pre;
  a.ld_pre = ld_pre;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.sw = sw_quant();
  a.ws = (uint8_t *)ws;
  a.wide_y = wide4(y, ldy, size_of(y_type)) && wide4(residual, ld_res, size_of(y_type));
  a.wide_pre = wide4(pre, ld_pre, 2);
  a.wide_bias = !bias || aligned(bias, 4 * size_of(bias_type));
  a.line_y = lines(y, ldy, size_of(y_type)) && lines(residual, ld_res, size_of(y_type));
  a.line_pre = lines(pre, ld_pre, 2);
  return hip_status(launch_linear(a, (hipStream_t)stream));
}

size_t mxfp4_linear_grad_pre_workspace_bytes(int64_t M, int64_t N) {
  return M < 1 || N < 1 || M > kMaxRows || N > kMaxRows ? 0 : grad_pre_workspace_bytes(M, N);
}

mxfp4_status_t mxfp4_linear_grad_pre(const void *dy, int dy_type, int64_t ld_dy, const void *pre, int64_t ld_pre,
                                     int activation, int gated, void *dz, int64_t ld_dz, float *dbias, int64_t M,
                                     int64_t N, void *workspace, size_t workspace_bytes, mxfp4_stream_t stream) {
  if (M < 0 || N < 1 || !known_act(activation) || !known_type(dy_type)) return MXFP4_ERR_INVALID_ARG;
  const bool needs_pre = gated || activation != MXFP4_ACT_NONE;
  if (M > 0 && (!dy || !dz || (needs_pre && !pre))) return MXFP4_ERR_INVALID_ARG;
  if (ld_dy < (gated ? N / 2 : N) || ld_dz < N || (needs_pre && ld_pre < N)) return MXFP4_ERR_INVALID_ARG;
  if (N % 16 != 0 || (gated && N % 32 != 0) || M > kMaxRows || N > kMaxRows || ld_dy > kMaxStride ||
      ld_dz > kMaxStride || (needs_pre && ld_pre > kMaxStride))
    return MXFP4_ERR_UNSUPPORTED;
  if (!aligned(dy, size_of(dy_type)) || !aligned(pre, 2) || !aligned(dz, 2) || !aligned(dbias, 4))
    return MXFP4_ERR_INVALID_ARG;
  if (M == 0 && !dbias) return MXFP4_OK;
  HeldWorkspace held;
  void *ws = nullptr;
  const mxfp4_status_t st = take_workspace(workspace, workspace_bytes, dbias ? grad_pre_workspace_bytes(M, N) : 0,
                                           (hipStream_t)stream, &held, &ws);
  if (st != MXFP4_OK) return st;
  GradPreArgs a{};
  a.dy = dy;
  a.dy_type = dy_type;
  a.ld_dy = ld_dy;
  a.pre = needs_pre ? (const uint16_t *)pre : nullptr;
  a.ld_pre = ld_pre;
  a.act = activation;
  a.gated = gated != 0;
  a.dz = (uint16_t *)dz;
  a.ld_dz = ld_dz;
  a.dbias = dbias;
  a.M = (int)M;
  a.N = (int)N;
  a.partial = (float *)ws;
  a.wide = wide4(dy, ld_dy, size_of(dy_type)) && wide4(a.pre, ld_pre, 2) && wide4(dz, ld_dz, 2);
  return hip_status(launch_grad_pre(a, (hipStream_t)stream));
}

size_t mxfp4_linear_grad_input_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M < 1 || N < 1 || K < 1 || !sizes_fit(M, N, K) ? 0 : grad_product_workspace_bytes(M, N, K, false);
}

mxfp4_status_t mxfp4_linear_grad_input(const void *dz, int64_t ld_dz, const void *Bq_sh, const void *Bs_sh, void *dx,
                                       int dx_type, int64_t ld_dx, int64_t M, int64_t N, int64_t K, void *workspace,
                                       size_t workspace_bytes, mxfp4_stream_t stream) {
  if (M < 0 || N < 1 || K < 1 || !known_type(dx_type)) return MXFP4_ERR_INVALID_ARG;
  if (!Bq_sh || !Bs_sh || (M > 0 && (!dz || !dx))) return MXFP4_ERR_INVALID_ARG;
  if (ld_dz < N || ld_dx < K) return MXFP4_ERR_INVALID_ARG;
  if (!sizes_fit(M, N, K) || !matrix_fits(N, K) || ld_dz > kMaxStride || ld_dx > kMaxStride)
    return MXFP4_ERR_UNSUPPORTED;
  if (!vector_rows(dz, ld_dz) || !aligned(Bq_sh, 16) || !aligned(Bs_sh, 16) || !aligned(dx, size_of(dx_type)))
    return MXFP4_ERR_INVALID_ARG;
  if (M == 0) return MXFP4_OK;
  HeldWorkspace held;
  void *ws = nullptr;
  const mxfp4_status_t st = take_workspace(workspace, workspace_bytes, grad_product_workspace_bytes(M, N, K, false),
                                           (hipStream_t)stream, &held, &ws);
  if (st != MXFP4_OK) return st;
  GradProductArgs a{};
  a.P = (const uint16_t *)dz;
  a.ldp = ld_dz;
  a.codes = (const uint8_t *)Bq_sh;
  a.scales = (const uint8_t *)Bs_sh;
  a.out = dx;
  a.out_type = dx_type;
  a.ld_out = ld_dx;
  a.I = (int)M;
  a.J = (int)N;
  a.K = (int)K;
  a.partial = (float *)ws;
  a.wide = lines(dx, ld_dx, size_of(dx_type));
  a.wide4 = wide4(dx, ld_dx, size_of(dx_type));
  return hip_status(launch_grad_product(a, (hipStream_t)stream));
}

size_t mxfp4_linear_grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M < 1 || N < 1 || K < 1 || !sizes_fit(M, N, K)
             ? 0
             : align256(packed_bytes(M, K)) + grad_product_workspace_bytes(N, M, K, true);
}

mxfp4_status_t mxfp4_linear_grad_weight(const void *dz, int64_t ld_dz, const void *x, int64_t ldx, void *dw,
                                        int dw_type, int64_t ld_dw, int64_t M, int64_t N, int64_t K, void *workspace,
                                        size_t workspace_bytes, mxfp4_stream_t stream) {
  if (M < 0 || N < 1 || K < 1 || !known_type(dw_type) || !dw || (M > 0 && (!dz || !x))) return MXFP4_ERR_INVALID_ARG;
  if (ld_dz < N || ldx < K || ld_dw < K) return MXFP4_ERR_INVALID_ARG;
  if (!sizes_fit(M, N, K) || ld_dz > kMaxStride || ldx > kMaxStride || ld_dw > kMaxStride) return MXFP4_ERR_UNSUPPORTED;
  if (!vector_rows(dz, ld_dz) || !vector_rows(x, ldx) || !aligned(dw, size_of(dw_type))) return MXFP4_ERR_INVALID_ARG;
  HeldWorkspace held;
  void *ws = nullptr;
  const size_t need = M > 0 ? align256(packed_bytes(M, K)) + grad_product_workspace_bytes(N, M, K, true) : 0;
  const mxfp4_status_t st = take_workspace(workspace, workspace_bytes, need, (hipStream_t)stream, &held, &ws);
  if (st != MXFP4_OK) return st;
  GradProductArgs a{};
  a.P = (const uint16_t *)dz;
  a.ldp = ld_dz;
  a.transposed = 1;
  a.out = dw;
  a.out_type = dw_type;
  a.ld_out = ld_dw;
  a.I = (int)N;
  a.J = (int)M;
  a.K = (int)K;
  a.wide = lines(dw, ld_dw, size_of(dw_type));
  a.wide4 = wide4(dw, ld_dw, size_of(dw_type));
  if (M > 0) {
    uint8_t *codes = (uint8_t *)ws, *scales = codes + align256(packed_codes_bytes(M, K));
    a.codes = codes;
    a.scales = scales;
    a.partial = (float *)(codes + align256(packed_bytes(M, K)));
    const hipError_t e = launch_pack_rows((const uint16_t *)x, ldx, M, K, codes, scales, sw_quant(), (hipStream_t)stream);
    if (e != hipSuccess) return hip_status(e);
  }
  return hip_status(launch_grad_product(a, (hipStream_t)stream));
}

}  // extern "C"
