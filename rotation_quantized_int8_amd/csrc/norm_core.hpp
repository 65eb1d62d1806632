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

}  // namespace convrot
