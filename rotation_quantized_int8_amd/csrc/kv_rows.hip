// Writing rows into the rotated, quantised key/value cache and reading them
// back (convrot_kv_append, convrot_kv_read).
//
// A row of D elements is held by L = D / 32 neighbouring lanes, four chunks of
// 8 elements each, chunk j L + lane: the lanes of a row touch neighbouring
// 16 bytes on its 16-bit side.  Of the log2 D butterfly stages of the
// rotation, five run in a lane's registers and the other one to three between
// lanes, by DPP permutations inside a 16-lane row (no LDS).
//
// A row costs 2 D bytes on its 16-bit side and D bits / 8 + 4 in the cache.
// Reading is bound by HBM: 65536 tokens of 8 heads of 128 from 4 bits take 69
// us, 4.9 TB/s where a large copy reaches 5.1.  Writing is bound by the vector
// unit next to it, about 22 operations an element of 4 cycles a wavefront
// (fp64 additions and conversions run at that rate too): 16384 tokens of 8
// heads of 128 in 8 bits 26.4 us, 3.9 TB/s.  1024 tokens of 16 heads in 4 bits
// take 6.3 and 4.8 us; four tokens of 8 heads 3.2 and 2.2 us, the latency of
// the loads.  The layout is what counted: with a lane's 64 bytes side by side instead of
// neighbouring lanes' 16 the large ones cost 38 and 94 us.  One pass over the
// rows, since a grid of 2048 workgroups that walks them reads the large
// context back in 95 us against 74; stores past the caches cost 77 us.

#include "kv.hpp"

namespace convrot {
namespace {

// The value of the lane whose number differs in bit BIT (0, 1 or 2).
template <int BIT>
__device__ __forceinline__ int lane_swap(int v) {
  if constexpr (BIT == 0) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);        // quad [1,0,3,2]
  else if constexpr (BIT == 1) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);   // quad [2,3,0,1]
  else {   // mirror the 8 lanes (i -> i ^ 7), then each quad (i -> i ^ 3)
    const int m = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
    return __builtin_amdgcn_update_dpp(0, m, 0x1B, 0xF, 0xF, true);
  }
}
template <int BIT>
__device__ __forceinline__ double lane_swap(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)lane_swap<BIT>((int)(uint32_t)u), hi = (uint32_t)lane_swap<BIT>((int)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// One stage between lanes: the lane with bit BIT clear keeps the sum, the
// other the difference (first minus second): v = other + sign * v.
template <int BIT>
__device__ __forceinline__ void stage_f64(double (&v)[32], int lane) {
  const double sign = (lane >> BIT) & 1 ? -1.0 : 1.0;
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = fma(v[i], sign, lane_swap<BIT>(v[i]));   // a product by +-1: one rounding
}
template <int BIT>
__device__ __forceinline__ void stage_i16(v2s (&v)[16], int lane) {
  const short sign = (lane >> BIT) & 1 ? -1 : 1;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    v[i] = v[i] * (v2s){sign, sign} + __builtin_bit_cast(v2s, lane_swap<BIT>(__builtin_bit_cast(int, v[i])));
}

// Codes of 32 values u with scale s, as 16 (4 bits) or 32 (8 bits) bytes.
// Rounds u / s half to even without dividing: r is within one ulp of 1 / s, so
// with low = r (1 - 3 2^-23) and high = r (1 + 3 2^-23), each rounded once, u /
// s and fp32(u / s) lie between u low and u high.  fma(x, y, 1.5 2^23) rounds
// the exact product half to even and leaves it in its low mantissa bits; where
// both ends round alike, so does all between.  Lanes where an element's ends
// differ (a half lies between: one in 3e5 / |u / s| elements), and scales
// whose reciprocal could leave fp32's normal range, divide.
template <int BITS>
__device__ __forceinline__ void codes32(const float (&u)[32], float s, uint32_t (&w)[BITS]) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
  const float r = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
  const float low = __fmul_rn(r, 1.0f - 0x3p-23f), high = __fmul_rn(r, 1.0f + 0x3p-23f);
  uint32_t b[32], apart = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    b[i] = __float_as_uint(__fmaf_rn(u[i], low, kMagic));
    const uint32_t other = __float_as_uint(__fmaf_rn(u[i], high, kMagic));
    asm("v_sad_u32 %0, %1, %2, %0" : "+v"(apart) : "v"(b[i]), "v"(other));   // += |b - other|
  }
  if (apart || s < 1e-30f || s > 1e30f) {
#pragma unroll
    for (int i = 0; i < 32; ++i) b[i] = __float_as_uint(__fadd_rn(s == 0.0f ? 0.0f : u[i] / s, kMagic));
  }
#pragma unroll
  for (int j = 0; j < BITS; ++j) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 32 / BITS; ++i) x = __builtin_amdgcn_alignbit(b[32 / BITS * j + i], x, BITS);   // in at the top
    w[j] = x;
  }
}

// blockIdx.y: 0 keys, 1 values.  The rotation runs in fp64, where the sums
// are exact (an fp16 value is a multiple of 2^-24 below 2^16, so a sum of 256
// of them has at most 48 significand bits).
template <int D, int BITS, bool BF16>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, KvRows kr, KvRows vr,
                                                        const int64_t* __restrict__ slots, int rows, KvDivider by_heads) {
  constexpr int L = D / 32;
  const KvRows in = blockIdx.y ? vr : kr;
  uint8_t* codes = blockIdx.y ? c.vc : c.kc;
  float* scales = blockIdx.y ? c.vs : c.ks;
  const int lane = threadIdx.x % L;
  const int per = 256 / L;
  for (uint32_t base = blockIdx.x * per; base < (uint32_t)rows; base += gridDim.x * per) {
    const uint32_t r = base + threadIdx.x / L;          // below 2^31 + 2^21
    const int t = (int)kv_divide(r, by_heads), h = (int)(r - (uint32_t)t * c.heads);
    int64_t slot = -1;
    v4u raw[4] = {};
    if (r < (uint32_t)rows) {   // dropped tokens too, so that the row does not wait for its slot
      slot = slots[t];
      const v4u* src = reinterpret_cast<const v4u*>(in.p + t * in.token + h * in.head) + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) raw[j] = src[j * L];
    }
    double v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t word = raw[i / 8][i / 2 % 4];
      v[i] = (double)in16_f32<BF16>(i & 1 ? word >> 16 : word & 0xFFFFu);
    }
#pragma unroll
    for (int k = 1; k < 32; k <<= 1)
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if ((i & k) == 0) {
          const double a = v[i], b = v[i + k];
          v[i] = a + b;
          v[i + k] = a - b;
        }
    stage_f64<0>(v, lane);
    if constexpr (L > 2) stage_f64<1>(v, lane);
    if constexpr (L > 4) stage_f64<2>(v, lane);
    // The largest |u| by its bits, where a NaN is above infinity.  An infinity or a NaN in a row leaves none of its u
    // finite, so that one u shows it; the others, and a u that passes fp32, are compared as numbers.
    float u[32], most = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = (float)v[i];
#pragma unroll
    for (int i = 0; i < 32; i += 2) most = fmaxf(fmaxf(most, fabsf(u[i])), fabsf(u[i + 1]));
    uint32_t top = max(__float_as_uint(most), __float_as_uint(u[0]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)lane_swap<0>((int)top));
    if constexpr (L > 2) top = max(top, (uint32_t)lane_swap<1>((int)top));
    if constexpr (L > 4) top = max(top, (uint32_t)lane_swap<2>((int)top));
    const bool finite = top < 0x7F800000u;
    const float s = __uint_as_float(top) / (BITS == 4 ? 7.0f : 127.0f);
    uint32_t w[BITS];
    codes32<BITS>(u, finite ? s : 0.0f, w);
    if (slot < 0 || slot >= c.slots) continue;
    const int64_t row = ((slot >> c.page_log2) * c.heads + h << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
    uint8_t* dst = codes + row * (D * BITS / 8) + lane * BITS;   // 8 codes are BITS bytes
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(dst + j * L * BITS) = finite ? w[j] : 0;
      else *reinterpret_cast<v2u*>(dst + j * L * BITS) = finite ? (v2u){w[2 * j], w[2 * j + 1]} : (v2u){0, 0};
    }
    if (lane == 0) scales[row] = finite ? __fmul_rn(s, kv_rsqrt(D)) : __uint_as_float(0x7FC00000u);
  }
}

// The codes' transform runs in packed 16-bit integers, where it is exact: a
// sum of 256 codes from -127 to 127 is at most 32512 in size.  Codes of -128,
// which kv_append does not write, fit too: the lowest sum is 256 times -128 =
// -32768 (of the row of W that has no minus), the highest 128 times 128 + 128
// times 127 = 32640.
template <int D, int BITS>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, const int64_t* __restrict__ slots, int rows,
                                                      KvDivider by_heads, uint16_t* ko, uint16_t* vo, int bf16) {
  constexpr int L = D / 32;
  const bool second = blockIdx.y || !ko;
  const uint8_t* codes = second ? c.vc : c.kc;
  const float* scales = second ? c.vs : c.ks;
  uint16_t* out = second ? vo : ko;
  const int lane = threadIdx.x % L;
  const int per = 256 / L;
  for (uint32_t base = blockIdx.x * per; base < (uint32_t)rows; base += gridDim.x * per) {
    const uint32_t r = base + threadIdx.x / L;          // below 2^31 + 2^21
    const int t = (int)kv_divide(r, by_heads), h = (int)(r - (uint32_t)t * c.heads);
    int64_t slot = r < (uint32_t)rows ? slots[t] : -1;
    if (slot >= c.slots) slot = -1;
    v4u raw[BITS / 4] = {};
    float f = 0.0f;
    if (slot >= 0) {
      const int64_t row = ((slot >> c.page_log2) * c.heads + h << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
      const uint8_t* src = codes + row * (D * BITS / 8) + lane * BITS;   // 8 codes are BITS bytes
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BITS == 4) {
          raw[0][j] = *reinterpret_cast<const uint32_t*>(src + j * L * BITS);
        } else {
          const v2u y = *reinterpret_cast<const v2u*>(src + j * L * BITS);
          raw[j / 2][2 * j % 4] = y[0], raw[j / 2][2 * j % 4 + 1] = y[1];
        }
      }
      f = __fmul_rn(scales[row], kv_rsqrt(D));
    }
    // v[i] holds two elements `gap` apart
    constexpr int gap = BITS == 4 ? 4 : 2;
    v2s v[16];
#pragma unroll
    for (int j = 0; j < BITS; ++j)
#pragma unroll
      for (int i = 0; i < gap; ++i) {
        const uint32_t x = raw[j / 4][j % 4] << (16 - BITS - BITS * i);
        v[gap * j + i] = __builtin_bit_cast(v2s, x) >> (v2s){16 - BITS, 16 - BITS};
      }
#pragma unroll
    for (int i = 0; i < 16; ++i) {   // the two halves: (a, b) -> (a + b, a - b)
      const uint32_t x = __builtin_bit_cast(uint32_t, v[i]);
      v[i] = v[i] * (v2s){1, -1} + __builtin_bit_cast(v2s, (x << 16) | (x >> 16));
    }
#pragma unroll
    for (int k = 1; k < 16; k <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i & k) == 0) {
          const v2s a = v[i], b = v[i + k];
          v[i] = a + b;
          v[i + k] = a - b;
        }
    stage_i16<0>(v, lane);
    if constexpr (L > 2) stage_i16<1>(v, lane);
    if constexpr (L > 4) stage_i16<2>(v, lane);
    if (r >= (uint32_t)rows) continue;
    v4u* dst = reinterpret_cast<v4u*>(out + (int64_t)r * D) + lane;
    // element e of the lane is in half e / gap % 2 of v[e / (2 gap) * gap + e % gap]
    uint32_t w[16];
    auto at = [&](int e) { return __fmul_rn((float)v[e / (2 * gap) * gap + e % gap][e / gap % 2], f); };
    if (bf16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2_rn(at(2 * i), at(2 * i + 1));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack_f16x2_rn(at(2 * i), at(2 * i + 1));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[j * L] = (v4u){w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
  }
}

// Workgroups of a launch over `rows` rows: one pass of the grid up to 8192
// workgroups (8 waves a SIMD on 256 CUs), then a stride.
unsigned row_grid(int64_t rows, int D) {
  const int64_t per = 256 / (D / 32), n = (rows + per - 1) / per;
  return (unsigned)(n < 8192 ? n : 8192);
}

template <int D, int BITS>
hipError_t append(const KvCache& c, const KvRows& k, const KvRows& v, bool bf16, const int64_t* slots, int64_t T,
                  hipStream_t stream) {
  const int rows = (int)(T * c.heads);
  const dim3 grid(row_grid(rows, D), 2);
  if (bf16) kv_append_kernel<D, BITS, true><<<grid, 256, 0, stream>>>(c, k, v, slots, rows, kv_divider((uint32_t)c.heads));
  else kv_append_kernel<D, BITS, false><<<grid, 256, 0, stream>>>(c, k, v, slots, rows, kv_divider((uint32_t)c.heads));
  return hipGetLastError();
}

template <int D, int BITS>
hipError_t read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* K, uint16_t* V, bool bf16,
                hipStream_t stream) {
  const int rows = (int)(T * c.heads);
  const dim3 grid(row_grid(rows, D), K && V ? 2 : 1);
  kv_read_kernel<D, BITS><<<grid, 256, 0, stream>>>(c, slots, rows, kv_divider((uint32_t)c.heads), K, V, bf16);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvCache& c, const KvRows& k, const KvRows& v, bool bf16, const int64_t* slots,
                            int64_t T, hipStream_t stream) {
  switch (c.head_dim * 16 + c.bits) {
    case 64 * 16 + 4: return append<64, 4>(c, k, v, bf16, slots, T, stream);
    case 64 * 16 + 8: return append<64, 8>(c, k, v, bf16, slots, T, stream);
    case 128 * 16 + 4: return append<128, 4>(c, k, v, bf16, slots, T, stream);
    case 128 * 16 + 8: return append<128, 8>(c, k, v, bf16, slots, T, stream);
    case 256 * 16 + 4: return append<256, 4>(c, k, v, bf16, slots, T, stream);
    default: return append<256, 8>(c, k, v, bf16, slots, T, stream);
  }
}

hipError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* K, uint16_t* V, bool bf16,
                          hipStream_t stream) {
  switch (c.head_dim * 16 + c.bits) {
    case 64 * 16 + 4: return read<64, 4>(c, slots, T, K, V, bf16, stream);
    case 64 * 16 + 8: return read<64, 8>(c, slots, T, K, V, bf16, stream);
    case 128 * 16 + 4: return read<128, 4>(c, slots, T, K, V, bf16, stream);
    case 128 * 16 + 8: return read<128, 8>(c, slots, T, K, V, bf16, stream);
    case 256 * 16 + 4: return read<256, 4>(c, slots, T, K, V, bf16, stream);
    default: return read<256, 8>(c, slots, T, K, V, bf16, stream);
  }
}

}  // namespace convrot
