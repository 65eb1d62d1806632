/*
 * convrot_mx.h -- C ABI of the rotated 4-bit linear for AMD MI355X (gfx950):
 * the linears of convrot.h with weights and activations in microscaled 4-bit
 * floating point (MXFP4: e2m1 elements, one power of two for 32 of them),
 * multiplied by the matrix cores as they are held.
 *
 * A row is rotated as in convrot.h, u = fp32(x H) in groups of 256 (fp64
 * butterflies: exact before the one rounding while a group's values span at
 * most 45 binades, fp16 always; fp32 weights 21 binades), and each block of 32
 * elements of u gets
 *   e = max(floor(log2(max|u|)) - 2, -127)     (-127 in a block of zeros)
 *   c = u 2^-e rounded to the nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties
 *       to even, beyond 6 to 6 (a sum of 0 is +0)
 * A block that holds an infinity or a NaN gets the scale NaN and codes of 0,
 * so it shows in every product with it.
 *
 * Layout.  codes [rows, K / 2] bytes, two codes a byte, the even element in the
 * low half (bit 3 the sign, bits 2..1 the exponent, bit 0 the mantissa).
 * scales [K / 256, rows, 8] bytes: block j of row r is e + 127 at
 * [j / 8, r, j % 8], 255 for NaN; the 8 scales of a rotation group side by
 * side, and those of neighbouring rows next to them, since that is how a tile
 * of the product reads them.
 *
 * Conventions are those of convrot.h: device pointers aligned to 16 bytes,
 * dense rows, caller-owned buffers, work enqueued on `stream` without
 * synchronising, all argument checks on the host before anything is enqueued,
 * errors as convrot_status.  K is a multiple of 256 (0 .. 131072), M and N are
 * 0 .. 2^24 with M N, M K and N K at most 2^35; with M = 0 or N = 0 nothing is
 * enqueued, with K = 0 a product is empty and Y the bias and the residual.
 */
#ifndef CONVROT_MX_H
#define CONVROT_MX_H

#include "convrot.h"

#ifdef __cplusplus
extern "C" {
#endif

/* W fp32 [N, K] -> codes and scales. */
convrot_status convrot_mx_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* codes, uint8_t* scales,
                                           void* stream);

/* X of `dtype` (convrot_dtype) [M, K] -> codes and scales. */
convrot_status convrot_mx_act_quant(const void* X, int dtype, int64_t M, int64_t K, uint8_t* codes,
                                    uint8_t* scales, void* stream);

/* The rows that codes and scales stand for, un-rotated: V [rows, K] of `dtype`
 * = out(fp32((c 2^e) H)), fp64 sums (exact while a group's values span at most 45
 * binades) and then two roundings, to fp32 as u has them and from there to the
 * type; the first changes nothing while the scales of a group lie within 2^12 of
 * one another.  A NaN scale gives NaN in its whole group. */
convrot_status convrot_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* V,
                                     int dtype, void* stream);

/* Y [M, N] of `dtype` = out(sum_k (c_x 2^e_x) (c_w 2^e_w) + bias + residual):
 * products on the matrix cores with fp32 sums, one rounding.  bias fp32 [N] or
 * NULL; residual [M, N] of `dtype` or NULL, which may be Y itself. */
convrot_status convrot_mx_gemm(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                               const uint8_t* w_scales, const float* bias, const void* residual, int64_t M,
                               int64_t N, int64_t K, void* Y, int dtype, void* stream);

/* Bytes of workspace of convrot_mx_linear (0 where it needs none), (size_t)-1
 * for invalid sizes. */
size_t convrot_mx_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* The whole linear: X [M, K] of `x_dtype` quantised as by convrot_mx_act_quant
 * into the workspace, then convrot_mx_gemm with Y of `y_dtype` (few short rows:
 * both in one launch, the same bits).  The workspace, which may be NULL where 0
 * bytes are needed, must not overlap anything, and calls that may run at the
 * same time need one each. */
convrot_status convrot_mx_linear(const void* X, int x_dtype, int64_t M, int64_t K, const uint8_t* w_codes,
                                 const uint8_t* w_scales, int64_t N, const float* bias, const void* residual,
                                 void* Y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_MX_H */
