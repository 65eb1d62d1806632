// C entry points of the rotated, quantised key/value cache: argument checks
// and launches.  Declarations and the full contract are in
// include/convrot_kv.h.

#include "checks.hpp"
#include "convrot_kv.h"
#include "kv.hpp"

using namespace convrot;

namespace {

constexpr int64_t kInt = 0x7FFFFFFF;

// Sizes of a cache, without its pointers.
bool cache_sizes_ok(const convrot_kv_cache* c) {
  return c->pages >= 1 && c->pages <= kInt && c->page_size >= CONVROT_KV_PAGE_MIN &&
         c->page_size <= CONVROT_KV_PAGE_MAX && (c->page_size & (c->page_size - 1)) == 0 && c->heads >= 1 &&
         c->heads <= 65535 && (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) &&
         (c->bits == 4 || c->bits == 8);
}

convrot_status check_cache(const convrot_kv_cache* c) {
  if (!c) return CONVROT_ERR_INVALID_ARG;
  if (!cache_sizes_ok(c)) return CONVROT_ERR_SHAPE;
  return CONVROT_OK;
}

convrot_status check_cache_pointers(const convrot_kv_cache* c) {
  if (!c->k_codes || !c->k_scale || !c->v_codes || !c->v_scale) return CONVROT_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scale) || !aligned16(c->v_codes) || !aligned16(c->v_scale))
    return CONVROT_ERR_ALIGNMENT;
  return CONVROT_OK;
}

KvCache view(const convrot_kv_cache* c) {
  KvCache v;
  v.kc = static_cast<uint8_t*>(c->k_codes);
  v.ks = c->k_scale;
  v.vc = static_cast<uint8_t*>(c->v_codes);
  v.vs = c->v_scale;
  v.slots = c->pages * c->page_size;
  v.pages = (int)c->pages;
  v.page_log2 = __builtin_ctzll((unsigned long long)c->page_size);
  v.heads = (int)c->heads;
  v.head_dim = (int)c->head_dim;
  v.bits = c->bits;
  return v;
}

// Does [p, p + n) touch one of the cache's four arrays?
bool meets_cache(const convrot_kv_cache* c, const void* p, size_t n) {
  const size_t rows = (size_t)c->pages * c->heads * c->page_size, cb = rows * (c->head_dim * c->bits / 8);
  return overlap(p, n, c->k_codes, cb) || overlap(p, n, c->v_codes, cb) || overlap(p, n, c->k_scale, rows * 4) ||
         overlap(p, n, c->v_scale, rows * 4);
}

bool strides_ok(int64_t token, int64_t head) {
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token <= kInt && head <= kInt;
}

// Bytes from the first to past the last element of [tokens, heads, D] rows.
size_t extent(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t D) {
  return (size_t)((tokens - 1) * token + (heads - 1) * head + D) * 2;
}

bool dtype_ok(int dtype) { return dtype == CONVROT_DTYPE_F16 || dtype == CONVROT_DTYPE_BF16; }

// The sizes of an attention call (the cache's own are checked before).
bool attention_sizes_ok(const convrot_kv_cache* c, int64_t T, int64_t q_heads, int64_t batch, int64_t max_q,
                        int64_t max_kv) {
  return T >= 0 && T <= kInt && batch >= 0 && batch <= 65535 && q_heads >= 1 && q_heads <= 65535 &&
         q_heads % c->heads == 0 && max_q >= 0 && max_q <= kInt && max_kv >= 0 && max_kv <= (1 << 30) &&
         max_q * (q_heads / c->heads) <= kInt - 4096;
}

KvAttn attention_args(const convrot_kv_cache* c, int64_t T, int64_t q_heads, int64_t batch, int64_t max_q,
                      int64_t max_kv) {
  KvAttn a{};
  a.c = view(c);
  a.T = T;
  a.batch = (int)batch;
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / c->heads);
  a.by_group = kv_divider((uint32_t)a.group);
  a.max_q = (int)(max_q < T ? max_q : T);
  a.max_kv = (int)max_kv;
  return a;
}

}  // namespace

extern "C" {

convrot_status convrot_kv_append(const convrot_kv_cache* cache, const void* K, int64_t k_token_stride,
                                 int64_t k_head_stride, const void* V, int64_t v_token_stride,
                                 int64_t v_head_stride, int dtype, const int64_t* slots, int64_t T, void* stream) {
  if (convrot_status st = check_cache(cache)) return st;
  if (T < 0 || T > kInt || T * cache->heads > kInt) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(dtype)) return CONVROT_ERR_INVALID_ARG;
  if (T == 0) return CONVROT_OK;
  if (!strides_ok(k_token_stride, k_head_stride) || !strides_ok(v_token_stride, v_head_stride))
    return CONVROT_ERR_SHAPE;
  if (!K || !V || !slots) return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_cache_pointers(cache)) return st;
  if (!aligned16(K) || !aligned16(V) || !aligned16(slots)) return CONVROT_ERR_ALIGNMENT;
  if (meets_cache(cache, K, extent(T, k_token_stride, cache->heads, k_head_stride, cache->head_dim)) ||
      meets_cache(cache, V, extent(T, v_token_stride, cache->heads, v_head_stride, cache->head_dim)) ||
      meets_cache(cache, slots, (size_t)T * 8))
    return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_device()) return st;
  const KvRows k{static_cast<const uint16_t*>(K), k_token_stride, k_head_stride};
  const KvRows v{static_cast<const uint16_t*>(V), v_token_stride, v_head_stride};
  return launched(launch_kv_append(view(cache), k, v, dtype == CONVROT_DTYPE_BF16, slots, T, as_stream(stream)));
}

convrot_status convrot_kv_read(const convrot_kv_cache* cache, const int64_t* slots, int64_t T, void* K, void* V,
                               int dtype, void* stream) {
  if (convrot_status st = check_cache(cache)) return st;
  if (T < 0 || T > kInt || T * cache->heads > kInt) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(dtype)) return CONVROT_ERR_INVALID_ARG;
  if (T == 0) return CONVROT_OK;
  if (!slots || (!K && !V)) return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_cache_pointers(cache)) return st;
  if (!aligned16(slots) || !aligned16(K) || !aligned16(V)) return CONVROT_ERR_ALIGNMENT;
  const size_t ob = (size_t)T * cache->heads * cache->head_dim * 2;
  if (meets_cache(cache, K, K ? ob : 0) || meets_cache(cache, V, V ? ob : 0) || overlap(K, ob, V, ob) ||
      overlap(K, ob, slots, (size_t)T * 8) || overlap(V, ob, slots, (size_t)T * 8))
    return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_device()) return st;
  return launched(launch_kv_read(view(cache), slots, T, static_cast<uint16_t*>(K), static_cast<uint16_t*>(V),
                                 dtype == CONVROT_DTYPE_BF16, as_stream(stream)));
}

size_t convrot_kv_workspace_bytes(const convrot_kv_cache* cache, int64_t T, int64_t q_heads, int64_t batch,
                                  int64_t max_q, int64_t max_kv) {
  if (!cache || !cache_sizes_ok(cache) || !attention_sizes_ok(cache, T, q_heads, batch, max_q, max_kv))
    return (size_t)-1;
  if (T == 0 || batch == 0 || max_q == 0) return 0;
  return kv_attention_workspace(attention_args(cache, T, q_heads, batch, max_q, max_kv));
}

convrot_status convrot_kv_attention(const convrot_kv_cache* cache, const void* Q, int64_t q_token_stride,
                                    int64_t q_head_stride, int dtype, int64_t T, int64_t q_heads,
                                    const int32_t* table, int64_t table_width, int64_t batch,
                                    const int32_t* kv_lens, const int32_t* q_start, int64_t max_q, int64_t max_kv,
                                    float sm_scale, int causal, void* O, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (convrot_status st = check_cache(cache)) return st;
  if (!attention_sizes_ok(cache, T, q_heads, batch, max_q, max_kv)) return CONVROT_ERR_SHAPE;
  if (table_width < 0 || table_width > kInt || max_kv > table_width * cache->page_size) return CONVROT_ERR_SHAPE;
  if (!dtype_ok(dtype)) return CONVROT_ERR_INVALID_ARG;
  if (T == 0) return CONVROT_OK;
  if (!q_start && (batch == 0 || T % batch || T / batch > max_q)) return CONVROT_ERR_SHAPE;
  if (batch == 0 || max_q == 0) return CONVROT_OK;
  if (!strides_ok(q_token_stride, q_head_stride)) return CONVROT_ERR_SHAPE;
  if (!Q || !O || !kv_lens || (table_width && !table)) return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_cache_pointers(cache)) return st;
  if (!aligned16(Q) || !aligned16(O) || !aligned16(kv_lens) || !aligned16(table) || !aligned16(q_start) ||
      !aligned16(workspace))
    return CONVROT_ERR_ALIGNMENT;
  KvAttn a = attention_args(cache, T, q_heads, batch, max_q, max_kv);
  const size_t need = kv_attention_workspace(a);
  if (need && (!workspace || workspace_bytes < need)) return CONVROT_ERR_WORKSPACE;
  const size_t ob = (size_t)T * q_heads * cache->head_dim * 2, tb = (size_t)batch * table_width * 4,
               lb = (size_t)batch * 4, sb = q_start ? lb + 4 : 0;
  const size_t qb = extent(T, q_token_stride, q_heads, q_head_stride, cache->head_dim);
  if (overlap(O, ob, Q, qb) || overlap(O, ob, table, tb) || overlap(O, ob, kv_lens, lb) ||
      overlap(O, ob, q_start, sb) || meets_cache(cache, O, ob) || overlap(workspace, need, O, ob) ||
      overlap(workspace, need, Q, qb) || overlap(workspace, need, table, tb) ||
      overlap(workspace, need, kv_lens, lb) || overlap(workspace, need, q_start, sb) ||
      meets_cache(cache, workspace, need))
    return CONVROT_ERR_INVALID_ARG;
  if (convrot_status st = check_device()) return st;
  a.q = KvRows{static_cast<const uint16_t*>(Q), q_token_stride, q_head_stride};
  a.o = static_cast<uint16_t*>(O);
  a.table = table;
  a.kv_lens = kv_lens;
  a.q_start = q_start;
  a.width = table_width;
  a.each_q = (int)(T / batch);
  a.scale = sm_scale;
  a.causal = causal != 0;
  a.bf16 = dtype == CONVROT_DTYPE_BF16;
  return launched(launch_kv_attention(a, workspace, as_stream(stream)));
}

}  // extern "C"
