// The rotated, quantised key/value cache: what its kernels share (internal to
// the library; the layout and arithmetic are stated in include/convrot_kv.h).
#pragma once

#include "common.hpp"

namespace convrot {

typedef short v2s __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// Division by a number the host knows: n / d = n * mul >> shift for n < 2^31.
// With l = ceil(log2 d), shift = 31 + l and mul = floor(2^shift / d) + 1 (below
// 2^32), the product overshoots 2^shift n / d by at most n < 2^31 <= 2^shift /
// d, so the quotient is exact.
struct KvDivider {
  uint32_t mul;
  int shift;
};
inline KvDivider kv_divider(uint32_t d) {
  KvDivider v{0, 31};
  while ((1ull << (v.shift - 31)) < d) ++v.shift;
  v.mul = (uint32_t)((1ull << v.shift) / d + 1);
  return v;
}
__device__ __forceinline__ uint32_t kv_divide(uint32_t n, KvDivider d) {
  return (uint32_t)((uint64_t)n * d.mul >> d.shift);
}

struct KvCache {
  uint8_t* kc;      // codes [pages, heads, page, D bits / 8]
  float* ks;        // scales [pages, heads, page]
  uint8_t* vc;
  float* vs;
  int64_t slots;    // pages * page
  int pages;
  int page_log2;
  int heads;
  int head_dim;
  int bits;
};

struct KvRows {     // 16-bit rows of D elements, [tokens, heads, D] with strides in elements
  const uint16_t* p;
  int64_t token, head;
};

struct KvAttn {
  KvCache c;
  KvRows q;
  uint16_t* o;            // [T, q_heads, D], dense
  const int* table;       // [batch, width]
  const int* kv_lens;     // [batch]
  const int* q_start;     // [batch + 1], or null: each_q queries a sequence
  int64_t T;
  int64_t width;
  int batch, q_heads, group;
  KvDivider by_group;
  int each_q;
  int max_q, max_kv;
  float scale;            // sm_scale
  int causal, bf16;
};

// The query that a row (query, head in group) belongs to.
__device__ __forceinline__ int kv_query_of(const KvAttn& a, int row) { return (int)kv_divide((uint32_t)row, a.by_group); }

hipError_t launch_kv_append(const KvCache& c, const KvRows& k, const KvRows& v, bool bf16, const int64_t* slots,
                            int64_t T, hipStream_t stream);
hipError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* K, uint16_t* V, bool bf16,
                          hipStream_t stream);
size_t kv_attention_workspace(const KvAttn& a);
hipError_t launch_kv_attention(const KvAttn& a, void* workspace, hipStream_t stream);

// fp32(D^-1/2)
__host__ __device__ constexpr float kv_rsqrt(int D) {
  return D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
}

template <bool BF16>
__device__ __forceinline__ float in16_f32(uint32_t bits) {
  if constexpr (BF16) return __uint_as_float(bits << 16);
  else return __half2float(__ushort_as_half((uint16_t)bits));
}

// Two fp32 values to bf16, each rounded once to nearest even, packed low then
// high (one v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16x2_rn(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){as_fp32(a), as_fp32(b)}, b2));
}

// The queries and tokens of a sequence, made safe: rows [first, first + n) lie
// in [0, T), and 0 <= kv <= max_kv.
struct KvSeq {
  int64_t first;
  int n, kv;
};
__device__ __forceinline__ KvSeq kv_safe(const KvAttn& a, int64_t from, int64_t to, int kv) {
  KvSeq s;
  from = from < 0 ? 0 : from > a.T ? a.T : from;
  to = to < from ? from : to > a.T ? a.T : to;
  s.first = from;
  s.n = to - from > a.max_q ? a.max_q : (int)(to - from);
  s.kv = kv < 0 ? 0 : kv > a.max_kv ? a.max_kv : kv;
  return s;
}
__device__ __forceinline__ KvSeq kv_sequence(const KvAttn& a, int b) {
  int64_t from = (int64_t)b * a.each_q, to = from + a.each_q;
  if (a.q_start) {
    from = a.q_start[b];
    to = a.q_start[b + 1];
  }
  return kv_safe(a, from, to, a.kv_lens[b]);
}

}  // namespace convrot
