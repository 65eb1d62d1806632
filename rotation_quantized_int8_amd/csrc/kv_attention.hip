// Attention over the rotated, quantised key/value cache.
//
// One wavefront per (query, query head): it rotates the query in LDS and
// walks over the visible tokens with the running maximum and sum of the
// softmax, D / 64 elements a lane.

#include "kv.hpp"

namespace convrot {
namespace {

// D floats in LDS times the +-1 matrix, by one wavefront.
template <int D>
__device__ __forceinline__ void rotate_lds(float* x, int lane) {
  for (int k = 1; k < D; k <<= 1) {
    float y[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int e = lane + 64 * i;
      y[i] = e & k ? x[e ^ k] - x[e] : x[e] + x[e ^ k];
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < D / 64; ++i) x[lane + 64 * i] = y[i];
    wave_lds_sync();
  }
}

template <int BITS>
__device__ __forceinline__ float code_at(const uint8_t* row, int e) {
  if constexpr (BITS == 8) return (float)(int8_t)row[e];
  else return (float)((int)((uint32_t)row[e / 2] << (e & 1 ? 24 : 28)) >> 28);
}

template <int D, int BITS>
__global__ __launch_bounds__(64) void kv_attention_kernel(KvAttn a) {
  constexpr int E = D / 64, ROW = D * BITS / 8;
  __shared__ float x[D];
  const int lane = threadIdx.x, h = blockIdx.y, i = blockIdx.x;
  const KvSeq s = kv_sequence(a, blockIdx.z);
  if (i >= s.n) return;
  const int64_t row = s.first + i;
  const uint16_t* q = a.q.p + row * a.q.token + h * a.q.head;
  for (int e = lane; e < D; e += 64) x[e] = a.bf16 ? in16_f32<true>(q[e]) : in16_f32<false>(q[e]);
  wave_lds_sync();
  rotate_lds<D>(x, lane);
  float qr[E], o[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) qr[e] = x[lane * E + e] * (a.scale * kv_rsqrt(D));
  wave_lds_sync();
  const int end = a.causal ? s.kv - s.n + i + 1 : s.kv, page = 1 << a.c.page_log2;
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j < end; ++j) {
    const int p = a.table[blockIdx.z * a.width + (j >> a.c.page_log2)];
    if (p < 0 || p >= a.c.pages) continue;
    const int64_t at = (((int64_t)p * a.c.heads + h / a.group) << a.c.page_log2) + (j & (page - 1));
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) dot += qr[e] * code_at<BITS>(a.c.kc + at * ROW, lane * E + e);
    for (int k = 32; k; k >>= 1) dot += __shfl_xor(dot, k);
    dot *= a.c.ks[at];
    const float top = fmaxf(m, dot), keep = expf(m - top), w = expf(dot - top);
    m = top;
    l = l * keep + w;
    const float wv = w * a.c.vs[at];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + wv * code_at<BITS>(a.c.vc + at * ROW, lane * E + e);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) x[lane * E + e] = l == 0.0f ? 0.0f : o[e] / l;
  wave_lds_sync();
  rotate_lds<D>(x, lane);
  for (int e = lane; e < D; e += 64)
    a.o[(row * a.q_heads + h) * D + e] = (uint16_t)out16(x[e] * kv_rsqrt(D), a.bf16);
}

template <int D, int BITS>
hipError_t attend(const KvAttn& a, hipStream_t stream) {
  kv_attention_kernel<D, BITS><<<dim3(a.max_q, a.q_heads, a.batch), 64, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const KvAttn&) { return 0; }

hipError_t launch_kv_attention(const KvAttn& a, void*, hipStream_t stream) {
  switch (a.c.head_dim * 16 + a.c.bits) {
    case 64 * 16 + 4: return attend<64, 4>(a, stream);
    case 64 * 16 + 8: return attend<64, 8>(a, stream);
    case 128 * 16 + 4: return attend<128, 4>(a, stream);
    case 128 * 16 + 8: return attend<128, 8>(a, stream);
    case 256 * 16 + 4: return attend<256, 4>(a, stream);
    default: return attend<256, 8>(a, stream);
  }
}

}  // namespace convrot
