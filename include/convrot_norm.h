/*
 * convrot_norm.h -- C ABI of the norms around the linears for AMD MI355X
 * (gfx950): the norm in front of a linear with its shift and scale, and the
 * gated residual behind it with the norm of the next, 16 bits out or rotated
 * and quantised for the linear that follows, in one pass over the rows.
 *
 * The norm of a row v [D], with its modulation's row i:
 *   n = ((v - mu) r weight + bias) (1 + scale_i) + shift_i
 *   mu = mean(v) (CONVROT_NORM_LAYER) or 0 (CONVROT_NORM_RMS)
 *   r  = (mean((v - mu)^2) + eps)^-1/2
 * The residual:
 *   h = residual_scale x + gate_i post(y)
 * with post a norm without modulation, or y itself; what follows takes h
 * before its rounding.  Outputs of 16 bits: all arithmetic is fp32 up to their
 * one rounding: the mean first, then the squares of the differences, with what
 * the mean's rounding left taken out (h itself is an fp32 number there).
 * Quantised outputs: all arithmetic is fp64 up to u = fp32(n H), so that codes
 * and scales are the formula's (H from h's fp32 value).  Rows of any finite size
 * have their norm (a row that fp32 does not hold is taken in fp64); an h that
 * passes fp32, an infinity or a NaN shows in its own row alone, as the formula
 * has it: a NaN in the whole row.
 *
 * Conventions are those of convrot.h, but for these.  Rows of X, Y and of the
 * modulation have strides in elements (0 .. 2^31 - 1) with D contiguous
 * elements each, and need no alignment but their element's; H and the outputs
 * are dense.  D is 1 .. 16384, for quantised outputs a multiple of 256; M is
 * 0 .. 2^24 with M D at most 2^35.
 */
#ifndef CONVROT_NORM_H
#define CONVROT_NORM_H

#include "convrot.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CONVROT_NORM_D_MAX 16384

enum { CONVROT_NORM_RMS = 1, CONVROT_NORM_LAYER = 2 };
enum { CONVROT_NORM_OUT_16 = 0, CONVROT_NORM_OUT_INT8 = 1, CONVROT_NORM_OUT_MXFP4 = 2 };
enum { CONVROT_NORM_DTYPE_F32 = 2 };   /* a modulation in fp32 (else its convrot_dtype) */

typedef struct convrot_norm_desc {
  int kind;              /* CONVROT_NORM_RMS or CONVROT_NORM_LAYER */
  float eps;             /* finite, at least 0 (below 2^-126 but not 0: 2^-126); with 0 a row without spread
                            gives NaN, as the formula does */
  const float* weight;   /* fp32 [D] or NULL (1) */
  const float* bias;     /* fp32 [D] or NULL (0) */
} convrot_norm_desc;

typedef struct convrot_modulation {
  const void* scale;     /* [rows, D] or NULL (0) */
  const void* shift;     /* [rows, D] or NULL (0) */
  const void* gate;      /* [rows, D] or NULL (1); read by convrot_residual_norm alone */
  int64_t scale_stride, shift_stride, gate_stride;
  int dtype;             /* of the three: the rows' dtype or CONVROT_NORM_DTYPE_F32 */
  int64_t rows;          /* at least 1 */
  const int32_t* index;  /* [M] the modulation's row of each row, or NULL: M / rows consecutive rows each, a
                            whole number.  A row whose index is out of 0 .. rows - 1 is not of any sequence:
                            nothing is written for it. */
} convrot_modulation;

typedef struct convrot_norm_out {
  int kind;              /* CONVROT_NORM_OUT_16: values [M, D] of the rows' dtype;
                            CONVROT_NORM_OUT_INT8: int8 codes [M, D] and fp32 scales [M] of n H as
                            convrot_act_quant gives them (a row with an infinity or a NaN: scale NaN, codes 0);
                            CONVROT_NORM_OUT_MXFP4: codes and scales of n H as convrot_mx_act_quant gives them */
  void* values;
  void* scales;
} convrot_norm_out;

/* X [M, D] of `dtype` (convrot_dtype) -> its norm.  mod may be NULL. */
convrot_status convrot_norm(const void* X, int64_t x_stride, int dtype, int64_t M, int64_t D,
                            const convrot_norm_desc* norm, const convrot_modulation* mod,
                            const convrot_norm_out* out, void* stream);

/* X and Y [M, D] -> H [M, D] (may be X or Y itself where that one is dense) and
 * the norm of h (norm and out NULL: H alone).  post NULL: y as it is. */
convrot_status convrot_residual_norm(const void* X, int64_t x_stride, const void* Y, int64_t y_stride, int dtype,
                                     int64_t M, int64_t D, float residual_scale, const convrot_norm_desc* post,
                                     const convrot_norm_desc* norm, const convrot_modulation* mod, void* H,
                                     const convrot_norm_out* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_NORM_H */
