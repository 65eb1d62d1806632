// C entry points of the norms around the linears: argument checks and
// launches.  Declarations and the full contract are in include/convrot_norm.h.

#include <cmath>

#include "checks.hpp"
#include "convrot_norm.h"
#include "norm.hpp"

using namespace convrot;

namespace {

constexpr int64_t kRowsMax = (int64_t)1 << 24, kElementsMax = (int64_t)1 << 35, kInt = 0x7FFFFFFF;

struct Range {
  const void* p;
  size_t bytes;
};

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Bytes from the first to past the last element of [rows, D] rows.
size_t extent(int64_t rows, int64_t stride, int64_t D, size_t size) {
  return rows > 0 ? (size_t)((rows - 1) * stride + D) * size : 0;
}

convrot_status check_desc(const convrot_norm_desc* d) {
  if (!d) return CONVROT_OK;
  if (d->kind != CONVROT_NORM_RMS && d->kind != CONVROT_NORM_LAYER) return CONVROT_ERR_INVALID_ARG;
  if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return CONVROT_ERR_INVALID_ARG;
  if (!aligned_to(d->weight, 4) || !aligned_to(d->bias, 4)) return CONVROT_ERR_ALIGNMENT;
  return CONVROT_OK;
}

// An eps in fp32's subnormals counts as the smallest normal number.
NormDesc view(const convrot_norm_desc* d) {
  if (!d) return NormDesc{kNormNone, 0.0f, nullptr, nullptr};
  const float eps = d->eps > 0.0f && d->eps < 0x1p-126f ? 0x1p-126f : d->eps;
  return NormDesc{d->kind, eps, d->weight, d->bias};
}

convrot_status run(const void* X, int64_t x_stride, const void* Y, int64_t y_stride, bool residual, int dtype,
                   int64_t M, int64_t D, float residual_scale, const convrot_norm_desc* post,
                   const convrot_norm_desc* norm, const convrot_modulation* mod, void* H,
                   const convrot_norm_out* out, void* stream) {
  if (M < 0 || M > kRowsMax || D < 1 || D > CONVROT_NORM_D_MAX || M * D > kElementsMax) return CONVROT_ERR_SHAPE;
  if (dtype != CONVROT_DTYPE_F16 && dtype != CONVROT_DTYPE_BF16) return CONVROT_ERR_INVALID_ARG;
  if (!norm != !out || (!residual && !norm)) return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_desc(post)) return st;
  if (convrot_status st = check_desc(norm)) return st;
  if (out) {
    if (out->kind < CONVROT_NORM_OUT_16 || out->kind > CONVROT_NORM_OUT_MXFP4) return CONVROT_ERR_INVALID_ARG;
    if (out->kind != CONVROT_NORM_OUT_16 && D % kGroup) return CONVROT_ERR_SHAPE;
  }
  if (x_stride < 0 || x_stride > kInt || y_stride < 0 || y_stride > kInt) return CONVROT_ERR_SHAPE;
  if (mod) {
    if (mod->rows < 1 || mod->rows > kRowsMax) return CONVROT_ERR_SHAPE;
    if (mod->scale_stride < 0 || mod->scale_stride > kInt || mod->shift_stride < 0 || mod->shift_stride > kInt ||
        mod->gate_stride < 0 || mod->gate_stride > kInt)
      return CONVROT_ERR_SHAPE;
    if (mod->dtype != dtype && mod->dtype != CONVROT_NORM_DTYPE_F32) return CONVROT_ERR_INVALID_ARG;
    if (!mod->index && M % mod->rows) return CONVROT_ERR_SHAPE;
  }
  if (M == 0) return CONVROT_OK;
  if (!X || (residual && (!Y || !H)) || (out && !out->values)) return CONVROT_ERR_INVALID_ARG;
  const bool quantised = out && out->kind != CONVROT_NORM_OUT_16;
  if (quantised && !out->scales) return CONVROT_ERR_INVALID_ARG;
  if (!aligned_to(X, 2) || !aligned_to(Y, 2) || !aligned_to(H, 2)) return CONVROT_ERR_ALIGNMENT;
  if (out && (!aligned_to(out->values, quantised ? 16 : 2) || (quantised && !aligned16(out->scales))))
    return CONVROT_ERR_ALIGNMENT;

  NormArgs a{};
  a.x = static_cast<const uint16_t*>(X);
  a.y = static_cast<const uint16_t*>(Y);
  a.x_stride = (uint32_t)x_stride;
  a.y_stride = (uint32_t)y_stride;
  a.M = (uint32_t)M;
  a.D = (int)D;
  a.residual_scale = residual_scale;
  a.post = view(post);
  a.norm = view(norm);
  a.h = static_cast<uint16_t*>(H);
  a.mod_rows = 1;
  a.inv_d = 1.0f / (float)D;
  a.inv_wide = 1.0 / (double)D;
  int64_t each = M;
  size_t mod_size = 2;
  if (mod) {
    mod_size = mod->dtype == CONVROT_NORM_DTYPE_F32 ? 4 : 2;
    if (!aligned_to(mod->scale, mod_size) || !aligned_to(mod->shift, mod_size) || !aligned_to(mod->gate, mod_size) ||
        !aligned_to(mod->index, 4))
      return CONVROT_ERR_ALIGNMENT;
    a.scale = mod->scale;
    a.shift = mod->shift;
    a.gate = residual ? mod->gate : nullptr;
    a.scale_stride = (uint32_t)mod->scale_stride;
    a.shift_stride = (uint32_t)mod->shift_stride;
    a.gate_stride = (uint32_t)mod->gate_stride;
    a.mod_f32 = mod_size == 4;
    a.mod_rows = (uint32_t)mod->rows;
    a.index = mod->index;
    each = mod->index ? 1 : M / mod->rows;
  }
  // r / each as a product: 2^31 each <= 2^shift, so the error of mul, below 1 in 2^shift / each, moves no r < 2^31
  a.each_shift = 31;
  while (((int64_t)1 << (a.each_shift - 31)) < each) ++a.each_shift;
  a.each_mul = (uint32_t)(((uint64_t)1 << a.each_shift) / (uint64_t)each + 1);
  if (out) {
    a.values = out->values;
    a.scales = out->scales;
  }

  // no output touches an input or another output, but H may be X or Y in place
  const size_t xb = extent(M, x_stride, D, 2), yb = residual ? extent(M, y_stride, D, 2) : 0;
  const int64_t B = a.mod_rows;
  const Range inputs[] = {
      {X, xb}, {Y, yb}, {a.post.weight, (size_t)D * 4}, {a.post.bias, (size_t)D * 4}, {a.norm.weight, (size_t)D * 4},
      {a.norm.bias, (size_t)D * 4}, {a.scale, extent(B, a.scale_stride, D, mod_size)},
      {a.shift, extent(B, a.shift_stride, D, mod_size)}, {a.gate, extent(B, a.gate_stride, D, mod_size)},
      {a.index, (size_t)M * 4}};
  size_t vb = 0, sb = 0;
  if (out) {
    vb = out->kind == CONVROT_NORM_OUT_16 ? (size_t)M * D * 2
         : out->kind == CONVROT_NORM_OUT_INT8 ? (size_t)M * D : (size_t)M * (D / 2);
    sb = out->kind == CONVROT_NORM_OUT_16 ? 0
         : out->kind == CONVROT_NORM_OUT_INT8 ? (size_t)M * 4 : (size_t)M * (D / kMxBlock);
  }
  const size_t hb = residual ? (size_t)M * D * 2 : 0;
  const bool x_in_place = X == H && (x_stride == D || M == 1), y_in_place = Y == H && (y_stride == D || M == 1);
  for (const Range& in : inputs) {
    if (overlap(a.values, vb, in.p, in.bytes) || overlap(a.scales, sb, in.p, in.bytes)) return CONVROT_ERR_INVALID_ARG;
    const bool in_place = (&in == &inputs[0] && x_in_place) || (&in == &inputs[1] && y_in_place);
    if (!in_place && overlap(H, hb, in.p, in.bytes)) return CONVROT_ERR_INVALID_ARG;
  }
  if (overlap(H, hb, a.values, vb) || overlap(H, hb, a.scales, sb) || overlap(a.values, vb, a.scales, sb))
    return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_device()) return st;
  const NormOut to = !out ? kOutNone : out->kind == CONVROT_NORM_OUT_16 ? kOut16
                                      : out->kind == CONVROT_NORM_OUT_INT8 ? kOutInt8 : kOutMx;
  return launched(launch_norm(a, dtype == CONVROT_DTYPE_BF16, to, as_stream(stream)));
}

}  // namespace

extern "C" {

convrot_status convrot_norm(const void* X, int64_t x_stride, int dtype, int64_t M, int64_t D,
                            const convrot_norm_desc* norm, const convrot_modulation* mod,
                            const convrot_norm_out* out, void* stream) {
  return run(X, x_stride, nullptr, 0, false, dtype, M, D, 1.0f, nullptr, norm, mod, nullptr, out, stream);
}

convrot_status convrot_residual_norm(const void* X, int64_t x_stride, const void* Y, int64_t y_stride, int dtype,
                                     int64_t M, int64_t D, float residual_scale, const convrot_norm_desc* post,
                                     const convrot_norm_desc* norm, const convrot_modulation* mod, void* H,
                                     const convrot_norm_out* out, void* stream) {
  return run(X, x_stride, Y, y_stride, true, dtype, M, D, residual_scale, post, norm, mod, H, out, stream);
}

}  // extern "C"
