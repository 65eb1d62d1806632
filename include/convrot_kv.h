/*
 * convrot_kv.h -- C ABI of the rotated, quantised key/value cache for AMD
 * MI355X (gfx950): the attention side of the INT8ConvRot linears in
 * convrot.h, with the same rotation and the same row quantisation.
 *
 * A row x of head_dim = D elements (one token, one head; a key or a value) is
 * held as
 *   u     = fp32(x W)           W the D x D Sylvester-Hadamard matrix of +-1;
 *                               the sum is exact before its one rounding (bf16
 *                               rows: while their values span <= 45 binades)
 *   s     = max|u| / qmax       an IEEE fp32 division; qmax = 7 (4 bits) or
 *                               127 (8 bits)
 *   c     = round_half_even(u / s) in [-qmax, qmax], 0 in a row of zeros
 *   scale = fp32(s * fp32(D^-1/2))
 * so (c scale) is the row in the orthonormal basis H = W D^-1/2 (symmetric,
 * HH = I) and (c scale) H the row itself.  A row that holds an infinity or a
 * NaN, or whose u passes fp32's range, gets scale = NaN and codes of 0, so
 * what reads it shows NaN.
 *
 * Layout.  The cache is paged.  codes [pages, heads, page_size, D bits / 8]
 * bytes and scales fp32 [pages, heads, page_size], one pair of arrays for the
 * keys and one for the values, dense.  4-bit codes are two's complement, two a
 * byte, the even element in the low half; 8-bit codes are int8 (-8 and -128,
 * which convrot_kv_append does not write, are read as such; scales are not
 * negative).  A slot is page * page_size + offset.
 *
 * Conventions are those of convrot.h: device pointers aligned to 16 bytes,
 * caller-owned buffers, work enqueued on `stream` without synchronising, all
 * argument checks on the host before anything is enqueued, errors as
 * convrot_status.  Slots, tables and lengths live on the device and are not
 * seen by the host: the kernels check them, and an entry that is out of range
 * reads and writes nothing (see each call).  Rows of K, V and Q are addressed
 * by a stride between tokens and one between heads, in elements, multiples of
 * 8 from 0 to 2^31 - 8; a row's D elements are contiguous.
 */
#ifndef CONVROT_KV_H
#define CONVROT_KV_H

#include "convrot.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CONVROT_KV_PAGE_MIN 16
#define CONVROT_KV_PAGE_MAX 256

typedef struct convrot_kv_cache {
  void* k_codes;     /* [pages, heads, page_size, head_dim * bits / 8] */
  float* k_scale;    /* [pages, heads, page_size] */
  void* v_codes;
  float* v_scale;
  int64_t pages;     /* at least 1, at most 2^31 - 1 */
  int64_t page_size; /* a power of two, 16 .. 256 */
  int64_t heads;     /* key/value heads, 1 .. 65535 */
  int64_t head_dim;  /* 64, 128 or 256 */
  int bits;          /* 4 or 8 */
} convrot_kv_cache;

/* Quantises T new tokens into their slots: K and V [T, heads, head_dim] of
 * `dtype` (convrot_dtype), slots int64 [T].  A slot below 0 or past the cache
 * drops its token (padding).  Two tokens of one call must not share a slot.
 * Only the tokens' own slots are written. */
convrot_status convrot_kv_append(const convrot_kv_cache* cache, const void* K, int64_t k_token_stride,
                                 int64_t k_head_stride, const void* V, int64_t v_token_stride,
                                 int64_t v_head_stride, int dtype, const int64_t* slots, int64_t T, void* stream);

/* Reads the rows of T slots back: K and V [T, heads, head_dim] of `dtype`,
 * dense, x = out(fp32(c W) * fp32(scale * fp32(D^-1/2))), where c W is exact.
 * Either of K and V may be NULL.  A slot out of range gives zeros. */
convrot_status convrot_kv_read(const convrot_kv_cache* cache, const int64_t* slots, int64_t T, void* K, void* V,
                               int dtype, void* stream);

/* Bytes of workspace that convrot_kv_attention needs for these sizes (0 where
 * it needs none), (size_t)-1 for invalid sizes. */
size_t convrot_kv_workspace_bytes(const convrot_kv_cache* cache, int64_t T, int64_t q_heads, int64_t batch,
                                  int64_t max_q, int64_t max_kv);

/* Attention over the cached rows of `batch` sequences, without un-rotating the
 * cache: O = softmax(sm_scale (q H) (c_k scale_k)^T) (c_v scale_v) H.
 *   Q, O      [T, q_heads, head_dim] of `dtype`; O dense.  q_heads is a
 *             multiple of cache->heads; query head h reads key head
 *             h / (q_heads / heads).
 *   q_start   int32 [batch + 1]: sequence b's queries are rows q_start[b] ..
 *             q_start[b + 1] - 1, at most max_q of them; NULL: T / batch each,
 *             a whole number and at most max_q.  Rows of no sequence are not
 *             written.
 *   kv_lens   int32 [batch]: cached tokens of each sequence, clamped to
 *             0 .. max_kv.
 *   table     int32 [batch, table_width]: token j of sequence b is at page
 *             table[b, j / page_size], offset j % page_size.  The tokens of a
 *             page number out of range are left out (an absent page).
 *   max_kv    at most table_width * page_size and 2^30.
 *   causal    nonzero: query i of n sees the first kv_len - n + i + 1 tokens
 *             (the queries are the sequence's last tokens, already cached);
 *             zero: every token (states of another length).
 * A query that sees no token gives zeros; a NaN scale shows in the queries
 * that see its token and in no other.  Sums, maxima and accumulators are fp32.
 * For up to 128 query rows (queries times heads of a group) per key head the
 * rotated queries enter the matrix cores as 16-bit fixed point of their row's
 * maximum and the scores are exact sums in int32; for more rows, after a power
 * of two of the row's own, fp16 queries enter as two fp16 numbers, bf16 queries
 * as one.  Either way a row is as exact next to any other.  A row whose
 * largest score passes 2^24 is taken with its scores scaled down to there, as
 * fp32 could not tell their differences apart.  The softmax weights enter
 * as fp16, at 2^8 and more for the largest, and for fp16 outputs of up to 128
 * rows as two fp16 numbers.  O must not overlap an input; the workspace (may
 * be NULL where 0 bytes are needed) must not overlap anything. */
convrot_status convrot_kv_attention(const convrot_kv_cache* cache, const void* Q, int64_t q_token_stride,
                                    int64_t q_head_stride, int dtype, int64_t T, int64_t q_heads,
                                    const int32_t* table, int64_t table_width, int64_t batch,
                                    const int32_t* kv_lens, const int32_t* q_start, int64_t max_q, int64_t max_kv,
                                    float sm_scale, int causal, void* O, void* workspace, size_t workspace_bytes,
                                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_KV_H */
