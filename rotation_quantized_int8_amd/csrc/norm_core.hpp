// Rows and modulations of the norms: loads, conversions and stores shared by
// their kernels (internal to the library).
#pragma once

#include "norm.hpp"

namespace convrot {

typedef uint16_t v8u __attribute__((ext_vector_type(8)));
typedef v8u v8u_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

// The modulation's row of a row; one out of range (negative ones too) is of no sequence.
__device__ __forceinline__ uint32_t mod_row(const NormArgs& a, uint32_t row) {
  return a.index ? (uint32_t)a.index[row] : (uint32_t)((uint64_t)row * a.each_mul >> a.each_shift);
}

template <bool kBF16>
__device__ __forceinline__ float widen(uint16_t b) {
  return kBF16 ? bf16_to_f32(b) : __half2float(__ushort_as_half(b));
}

// 8 values to the rows' type, nearest even.
template <bool kBF16>
__device__ __forceinline__ v8u narrow(const float (&v)[8]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = kBF16 ? __builtin_bit_cast(int, __builtin_convertvector((f2){v[2 * i], v[2 * i + 1]}, b2))
                 : (int)pack_f16x2_rn(v[2 * i], v[2 * i + 1]);
  return __builtin_bit_cast(v8u, r);
}

// 8 neighbouring elements from e0 of a 16-bit row of D (zeros past its end).
// kWhole: the chunk lies wholly inside the row, or wholly outside.
template <bool kWhole>
__device__ __forceinline__ v8u load8(const uint16_t* row, int e0, int D) {
  if (kWhole ? e0 < D : e0 + 8 <= D) return *reinterpret_cast<const v8u_any*>(row + e0);
  v8u v = {0, 0, 0, 0, 0, 0, 0, 0};
  if constexpr (!kWhole) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i < D) v[i] = row[e0 + i];
  }
  return v;
}
template <bool kWhole>
__device__ __forceinline__ void load8(const float* row, int e0, int D, float (&f)[8]) {
  if (kWhole || e0 + 8 <= D) {
    const v4f a = *reinterpret_cast<const v4f_any*>(row + e0), b = *reinterpret_cast<const v4f_any*>(row + e0 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e0 + i < D ? row[e0 + i] : 0.0f;
  }
}
// The same of a modulation's row.
template <bool kBF16, bool kWhole>
__device__ __forceinline__ void load_mod(const void* base, int64_t at, int f32, int e0, int D, float (&f)[8]) {
  if (f32) {
    load8<kWhole>(static_cast<const float*>(base) + at, e0, D, f);
  } else {
    const v8u v = load8<kWhole>(static_cast<const uint16_t*>(base) + at, e0, D);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = widen<kBF16>(v[i]);
  }
}
template <bool kWhole>
__device__ __forceinline__ void store8(uint16_t* row, int e0, int D, v8u v) {
  if (kWhole || e0 + 8 <= D) {
    *reinterpret_cast<v8u_any*>(row + e0) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i < D) row[e0 + i] = v[i];
  }
}

// Statistics in fp64.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double joined(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wavefront, the same bits in every lane.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  uint64_t b = __builtin_bit_cast(uint64_t, v);
  uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
  const auto l16 = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  const auto h16 = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  v = joined(l16[0], h16[0]) + joined(l16[1], h16[1]);
  b = __builtin_bit_cast(uint64_t, v);
  lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
  const auto l32 = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  const auto h32 = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  return joined(l32[0], h32[0]) + joined(l32[1], h32[1]);
}

// Sum over the row's wavefronts, in their order.  `part` is written by this sum
// alone until the next barrier has passed.
template <int WAVES>
__device__ __forceinline__ double row_sum(double v, double* part) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[w];
  }
  return v;
}
// v^-1/2: the hardware's estimate (some 24 bits) and two Newton steps; 0 for an
// infinity, an infinity for 0.
__device__ __forceinline__ double inverse_root(double v) {
  const double y0 = __builtin_amdgcn_rsq(v);
  double y = y0;
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __fma_rn(0.5 * y, __fma_rn(-v * y, y, 1.0), y);
  return y0 > 0.0 && y0 < __builtin_inf() ? y : y0;
}

// s / d, with inv 1 / d: a product, and what it is off.  The sum of d equal values gives the value.
__device__ __forceinline__ double quotient(double s, double d, double inv) {
  const double v = s * inv;
  return __fma_rn(__fma_rn(-v, d, s), inv, v);
}

}  // namespace convrot
