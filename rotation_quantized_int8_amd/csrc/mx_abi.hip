// C entry points of the rotated 4-bit linear: argument checks and launches.
// Declarations and the full contract are in include/convrot_mx.h.

#include "checks.hpp"
#include "convrot_mx.h"
#include "mx.hpp"

using namespace convrot;

namespace {

constexpr int64_t kRowsMax = (int64_t)1 << 24, kElementsMax = (int64_t)1 << 35;

bool k_ok(int64_t K) { return K >= 0 && K % kGroup == 0 && K <= kKMax; }
bool rows_ok(int64_t rows, int64_t K) { return rows >= 0 && rows <= kRowsMax && rows * K <= kElementsMax; }
bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return k_ok(K) && rows_ok(M, K) && rows_ok(N, K) && M * N <= kElementsMax;
}
bool dtype_ok(int dtype) { return dtype == CONVROT_DTYPE_F16 || dtype == CONVROT_DTYPE_BF16; }
size_t codes_bytes(int64_t rows, int64_t K) { return (size_t)rows * (K / 2); }
size_t scales_bytes(int64_t rows, int64_t K) { return (size_t)rows * (K / kMxBlock); }

// One tensor of a quantiser: [rows, K] on one side, codes and scales on the other.
convrot_status check_rows(const void* V, size_t v_bytes, const void* codes, const void* scales, int64_t rows,
                          int64_t K) {
  if (!V || !codes || !scales) return CONVROT_ERR_INVALID_ARG;
  if (!aligned16(V) || !aligned16(codes) || !aligned16(scales)) return CONVROT_ERR_ALIGNMENT;
  const size_t cb = codes_bytes(rows, K), sb = scales_bytes(rows, K);
  if (overlap(V, v_bytes, codes, cb) || overlap(V, v_bytes, scales, sb) || overlap(codes, cb, scales, sb))
    return CONVROT_ERR_INVALID_ARG;
  return check_device();
}

// The product's operands and output but the activations (codes, or X of the
// whole linear), which are the caller's inputs a and b.
convrot_status check_product(const void* a, size_t ab, const void* b, size_t bb, const void* w_codes,
                             const void* w_scales, const float* bias, const void* residual, int64_t M, int64_t N,
                             int64_t K, const void* Y) {
  if (!Y || (K && (!a || !w_codes || !w_scales))) return CONVROT_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(bias) ||
      !aligned16(residual) || !aligned16(Y))
    return CONVROT_ERR_ALIGNMENT;
  const size_t yb = (size_t)M * N * 2;
  if (overlap(Y, yb, a, ab) || overlap(Y, yb, b, bb) || overlap(Y, yb, w_codes, codes_bytes(N, K)) ||
      overlap(Y, yb, w_scales, scales_bytes(N, K)) || overlap(Y, yb, bias, (size_t)N * 4) ||
      (residual != Y && overlap(Y, yb, residual, yb)))
    return CONVROT_ERR_INVALID_ARG;
  return CONVROT_OK;
}

}  // namespace

extern "C" {

convrot_status convrot_mx_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* codes, uint8_t* scales,
                                           void* stream) {
  if (!k_ok(K) || !rows_ok(N, K)) return CONVROT_ERR_SHAPE;
  if (N == 0 || K == 0) return CONVROT_OK;
  if (convrot_status st = check_rows(W, (size_t)N * K * 4, codes, scales, N, K)) return st;
  return launched(launch_mx_quantize_weights(W, N, K, codes, scales, as_stream(stream)));
}

convrot_status convrot_mx_act_quant(const void* X, int dtype, int64_t M, int64_t K, uint8_t* codes,
                                    uint8_t* scales, void* stream) {
  if (!k_ok(K) || !rows_ok(M, K)) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(dtype)) return CONVROT_ERR_INVALID_ARG;
  if (M == 0 || K == 0) return CONVROT_OK;
  if (convrot_status st = check_rows(X, (size_t)M * K * 2, codes, scales, M, K)) return st;
  return launched(launch_mx_act_quant(X, dtype == CONVROT_DTYPE_BF16, M, K, codes, scales, as_stream(stream)));
}

convrot_status convrot_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* V,
                                     int dtype, void* stream) {
  if (!k_ok(K) || !rows_ok(rows, K)) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(dtype)) return CONVROT_ERR_INVALID_ARG;
  if (rows == 0 || K == 0) return CONVROT_OK;
  if (convrot_status st = check_rows(V, (size_t)rows * K * 2, codes, scales, rows, K)) return st;
  return launched(launch_mx_dequantize(codes, scales, rows, K, V, dtype == CONVROT_DTYPE_BF16, as_stream(stream)));
}

convrot_status convrot_mx_gemm(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                               const uint8_t* w_scales, const float* bias, const void* residual, int64_t M,
                               int64_t N, int64_t K, void* Y, int dtype, void* stream) {
  if (!sizes_ok(M, N, K)) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(dtype)) return CONVROT_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return CONVROT_OK;
  if (K && !x_scales) return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_product(x_codes, codes_bytes(M, K), x_scales, scales_bytes(M, K), w_codes, w_scales,
                                        bias, residual, M, N, K, Y))
    return st;
  if (convrot_status st = check_device()) return st;
  return launched(launch_mx_gemm(MxGemm{x_codes, x_scales, w_codes, w_scales, bias, residual, Y, M, N, K,
                                        dtype == CONVROT_DTYPE_BF16, 1},
                                 as_stream(stream)));
}

size_t convrot_mx_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!sizes_ok(M, N, K)) return (size_t)-1;
  return M == 0 || N == 0 || mx_fusable(M, N, K) ? 0 : round256(codes_bytes(M, K)) + round256(scales_bytes(M, K));
}

convrot_status convrot_mx_linear(const void* X, int x_dtype, int64_t M, int64_t K, const uint8_t* w_codes,
                                 const uint8_t* w_scales, int64_t N, const float* bias, const void* residual,
                                 void* Y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(M, N, K)) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return CONVROT_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return CONVROT_OK;
  const size_t xb = (size_t)M * K * 2, need = convrot_mx_workspace_bytes(M, N, K), yb = (size_t)M * N * 2;
  if (convrot_status st = check_product(X, xb, nullptr, 0, w_codes, w_scales, bias, residual, M, N, K, Y)) return st;
  if (!aligned16(workspace)) return CONVROT_ERR_ALIGNMENT;
  if (need && (!workspace || workspace_bytes < need)) return CONVROT_ERR_WORKSPACE;
  if (overlap(workspace, need, X, xb) || overlap(workspace, need, w_codes, codes_bytes(N, K)) ||
      overlap(workspace, need, w_scales, scales_bytes(N, K)) || overlap(workspace, need, bias, (size_t)N * 4) ||
      overlap(workspace, need, residual, yb) || overlap(workspace, need, Y, yb))
    return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_device()) return st;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + round256(codes_bytes(M, K));
  const MxGemm a{codes, scales, w_codes, w_scales, bias, residual, Y, M, N, K, y_dtype == CONVROT_DTYPE_BF16, 1};
  if (mx_fusable(M, N, K)) return launched(launch_mx_fused(a, X, x_dtype == CONVROT_DTYPE_BF16, as_stream(stream)));
  if (K) {
    const hipError_t e =
        launch_mx_act_quant(X, x_dtype == CONVROT_DTYPE_BF16, M, K, codes, scales, as_stream(stream));
    if (e != hipSuccess) return CONVROT_ERR_LAUNCH;
  }
  return launched(launch_mx_gemm(a, as_stream(stream)));
}

}  // extern "C"
