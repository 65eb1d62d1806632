// Microscaled 4-bit floating point: the device pieces that every quantiser
// shares, and the launchers (internal to the library).
#pragma once

#include "launch.hpp"
#include "rotate.hpp"

namespace convrot {

constexpr int kMxBlock = 32;

// Rotation of a group whose row `lane` (elements 16 lane .. + 15) this lane
// holds in fp32, in place: along the row in registers, a transpose in the
// segment's LDS slot (16-byte chunks swizzled by row, conflict-free both ways),
// along the column, and the transpose back.  The transform is that of +-1: what it
// leaves is 16 u.
constexpr int kTurnSlot = 1024 + 64;   // bytes: 256 floats, and an offset of 16 banks to the next slot
__device__ __forceinline__ void fwht16(float (&v)[16]) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
}
__device__ __forceinline__ void rotate_rows(float (&v)[16], char* slot, int lane) {
  const int key = (lane >> 2) & 3;
  fwht16(v);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<float4*>(slot + 64 * lane + 16 * (c ^ key)) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  wave_lds_sync();
  float* sf = reinterpret_cast<float*>(slot) + (lane & 3);
#pragma unroll
  for (int a = 0; a < 16; ++a) v[a] = sf[16 * a + 4 * (key ^ (a >> 2))];
  wave_lds_sync();
  fwht16(v);
#pragma unroll
  for (int a = 0; a < 16; ++a) sf[16 * a + 4 * (key ^ (a >> 2))] = v[a];
  wave_lds_sync();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 t = *reinterpret_cast<const float4*>(slot + 64 * lane + 16 * (c ^ key));
    v[4 * c] = t.x;
    v[4 * c + 1] = t.y;
    v[4 * c + 2] = t.z;
    v[4 * c + 3] = t.w;
  }
  wave_lds_sync();
}

// The same in fp64 (kSlotBytes), rounded once to fp32: f[] holds fp32(16 v H).
__device__ __forceinline__ void rotate_rows(double (&v)[16], char* slot, int lane, float (&f)[16]) {
  fwht16(v);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<double2*>(slot + 128 * lane + 16 * (q ^ (lane & 7))) = make_double2(v[2 * q], v[2 * q + 1]);
  wave_lds_sync();
  const double* sd = reinterpret_cast<const double*>(slot);
#pragma unroll
  for (int a = 0; a < 16; ++a) v[a] = sd[16 * a + 2 * ((lane >> 1) ^ (a & 7)) + (lane & 1)];
  wave_lds_sync();
  fwht16(v);
  float* sf = reinterpret_cast<float*>(slot) + (lane & 3);
  const int key = (lane >> 2) & 3;
#pragma unroll
  for (int a = 0; a < 16; ++a) sf[16 * a + 4 * (key ^ (a >> 2))] = (float)v[a];
  wave_lds_sync();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 r = *reinterpret_cast<const float4*>(slot + 64 * lane + 16 * (c ^ key));
    f[4 * c] = r.x;
    f[4 * c + 1] = r.y;
    f[4 * c + 2] = r.z;
    f[4 * c + 3] = r.w;
  }
  wave_lds_sync();
}

// The rotated values of an activation group from rotate_group's 16 u: fp16 keeps
// the factor 2^4 (16 u stays in fp32's normal range) and gives it to the scale;
// bf16 takes u itself, which may be as large or small as fp32 holds.  The sum
// with 0 makes a zero +0.
__host__ __device__ constexpr int mx_up(bool bf16) { return bf16 ? 0 : 4; }
template <bool kBF16>
__device__ __forceinline__ void mx_rotated(const double (&y)[16], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = kBF16 ? (float)__fma_rn(y[i], 0.0625, 0.0) : (float)y[i] + 0.0f;
}

// Scale byte of the block of 32 that this lane and its neighbour (lane ^ 1)
// hold 16 elements each of; kUp: f is 2^kUp times the value quantised.
template <int kUp>
__device__ __forceinline__ uint32_t mx_scale_byte(const float (&f)[16]) {
  // the bits order like |f| within a sign, NaN on top: the largest as signed numbers is of the positive values, as
  // unsigned ones of the negative, if there are any (three at a time, without clearing signs)
  int pos = 0;
  uint32_t neg = 0;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    pos = max(max(pos, __float_as_int(f[i])), __float_as_int(f[i + 1]));
    neg = max(max(neg, __float_as_uint(f[i])), __float_as_uint(f[i + 1]));
  }
  uint32_t m = max((uint32_t)pos, neg & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
  const int eb = (int)(m >> 23);
  return eb == 255 ? 255u : (uint32_t)max(eb - 2 - kUp, 0);
}

// The lane's 16 codes, 8 bytes.  The conversion takes its scale as the
// exponent field of an fp32 number, so 2^(byte - 127) is byte << 23, also for
// byte 0; it rounds to nearest, ties to even, and saturates.
template <int kUp>
__device__ __forceinline__ uint2 mx_codes(const float (&f)[16], uint32_t byte) {
  const float s = __uint_as_float((byte + kUp) << 23);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], f[8 * j], f[8 * j + 1], s, 0);
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], f[8 * j + 2], f[8 * j + 3], s, 1);
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], f[8 * j + 4], f[8 * j + 5], s, 2);
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], f[8 * j + 6], f[8 * j + 7], s, 3);
  }
  return byte == 255u ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

// Quantises the lane's 16 elements of group g of a row and stores codes and
// scale (one byte by the even lane of a block).
template <int kUp>
__device__ __forceinline__ void mx_store(const float (&f)[16], int64_t row, int64_t rows, int64_t K, int64_t g,
                                         int lane, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint32_t byte = mx_scale_byte<kUp>(f);
  *reinterpret_cast<uint2*>(codes + row * (K / 2) + g * 128 + 8 * lane) = mx_codes<kUp>(f, byte);
  if ((lane & 1) == 0) scales[(g * rows + row) * 8 + (lane >> 1)] = (uint8_t)byte;
}

struct MxGemm {
  const uint8_t *x, *xs, *w, *ws;   // codes [M, K / 2] and [N, K / 2], scales [K / 256, rows, 8]
  const float* bias;                // [N] or null
  const void* res;                  // [M, N] of the output's type or null (may be out)
  void* out;                        // [M, N]
  int64_t M, N, K;
  int bf16;                         // output (and residual) bf16 instead of fp16
  int64_t group_m;                  // row tiles per group of the tile order (set by the launcher)
};

hipError_t launch_mx_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* codes, uint8_t* scales,
                                      hipStream_t stream);
hipError_t launch_mx_act_quant(const void* X, bool bf16, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* V,
                                bool bf16, hipStream_t stream);
hipError_t launch_mx_gemm(const MxGemm& a, hipStream_t stream);
// The whole linear in one launch for few short rows: a.x and a.xs are unused, X
// is the activation [M, K].
bool mx_fusable(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_fused(const MxGemm& a, const void* X, bool bf16, hipStream_t stream);

}  // namespace convrot
