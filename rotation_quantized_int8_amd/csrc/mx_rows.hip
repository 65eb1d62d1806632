// Rows to microscaled 4-bit floating point and back: weights (fp32) and
// activations (fp16, bf16) rotated and quantised, and the rows that codes and
// scales stand for.
//
// Mathematics.  u = fp32(x H) in groups of 256; a block of 32 has the scale
// 2^e, e = max(floor(log2 max|u|) - 2, -127), so that its largest value lies in
// [4, 8) of the codes' +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} (those past 6 saturate).
// floor(log2) is the exponent field of the maximum's bits; the codes come from
// the hardware conversion, which rounds to nearest even.
//
// Work split.  As in the int8 prologue 16 lanes own a group of 256, each the 16
// elements of one row of the 16 x 16 view, so a block of 32 is two neighbouring
// lanes: one lane permutation completes its maximum.  No scale spans a row, so
// groups are independent and no workgroup barrier is needed.  A workgroup's 16
// groups are the same one of 16 neighbouring rows, whose scales are one line of 128
// bytes (16 groups of one row write 16 pieces of 8 bytes, 18 % more to memory; times
// level to 4 %).
//
// Bound and measured (us, one call after another in a graph, inputs in turn; a call
// traced alone takes 1 to 4 more).  Activations: 8192 x 8192 44 (3.9 TB/s), 16384 x
// 2048 22, 1024 x 8192 7.5; one group a workgroup and no loads ahead are 15 % slower.
// The vector unit is 60 % busy and memory three quarters: the slots leave 4
// wavefronts a SIMD, which wait for LDS and loads in turn (sums in fp32 where they
// are certain are level, so their width is not what bounds it).  Weights by memory:
// 8192 x 2048 14.8 (5.2 TB/s).  Values back by memory: 16384 x 2048 18.5 (4.6 TB/s),
// in fp64 36.

#include "mx.hpp"

namespace convrot {
namespace {

constexpr int kSegs = 16;   // groups of a 256-thread workgroup

// The groups of [rows, K]: 16 rows at a time, group after group (fewer than 2^31,
// so n / (16 G) is a product; only the last rows, if there are not 16, divide).
struct Units {
  uint32_t rows, G, total, mul;
  int shift;
};
__device__ __forceinline__ void unit_of(const Units& t, uint32_t u, uint32_t& row, uint32_t& g) {
  const uint32_t block = (uint32_t)((uint64_t)u * t.mul >> t.shift), in = u - block * 16u * t.G;
  const uint32_t left = t.rows - 16u * block;
  g = left >= 16u ? in >> 4 : in / left;
  row = 16u * block + (left >= 16u ? in & 15u : in - g * left);
}
Units units(int64_t rows, int64_t K) {
  Units t{(uint32_t)rows, (uint32_t)(K / kGroup), (uint32_t)(rows * (K / kGroup)), 0u, 31};
  const uint64_t d = 16ull * t.G;
  while ((1ull << (t.shift - 31)) < d) ++t.shift;
  t.mul = (uint32_t)((1ull << t.shift) / d + 1);
  return t;
}

// A workgroup whose grid does not cover all groups takes every gridDim-th 16 and
// has the next ones' loads in flight while it works on these.
template <bool kBF16>
__global__ void __launch_bounds__(256)
mx_act_quant_kernel(const uint16_t* __restrict__ X, int64_t K, Units t, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales) {
  __shared__ __align__(16) char smem[kSegs * kSlotBytes];
  const int seg = threadIdx.x >> 4, lane = threadIdx.x & 15;
  uint32_t u = blockIdx.x * kSegs + seg, row, g;
  if (u >= t.total) return;
  auto source = [&](uint32_t row, uint32_t g) {
    return reinterpret_cast<const v4i*>(X + row * K + g * kGroup + 16 * lane);
  };
  unit_of(t, u, row, g);
  const v4i* src = source(row, g);
  v4i r0 = src[0], r1 = src[1];
  char* slot = smem + seg * kSlotBytes;
  for (;;) {
    const uint32_t next = u + gridDim.x * kSegs;
    const bool more = next < t.total;
    uint32_t next_row = 0, next_g = 0;
    park_row(slot, lane, r0, r1);
    if (more) {
      unit_of(t, next, next_row, next_g);
      src = source(next_row, next_g);
      r0 = src[0];
      r1 = src[1];
    }
    double y[16];
    float f[16];
    rotate_staged<kBF16>(slot, lane, y);
    mx_rotated<kBF16>(y, f);
    mx_store<mx_up(kBF16)>(f, row, t.rows, K, g, lane, codes, scales);
    if (!more) return;
    u = next;
    row = next_row;
    g = next_g;
  }
}

__global__ void __launch_bounds__(256)
mx_quantize_weights_kernel(const float* __restrict__ W, int64_t K, Units t, uint8_t* __restrict__ codes,
                           uint8_t* __restrict__ scales) {
  __shared__ __align__(16) char smem[kSegs * kSlotBytes];
  const int seg = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const uint32_t u = blockIdx.x * kSegs + seg;
  if (u >= t.total) return;
  uint32_t row, g;
  unit_of(t, u, row, g);
  const v4f* src = reinterpret_cast<const v4f*>(W + row * K + g * kGroup + 16 * lane);
  double v[16];   // the sum with 0 makes a zero +0, and so every zero after it
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const v4f w = src[c];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * c + i] = __fma_rn((double)w[i], 0.0625, 0.0);
  }
  float f[16];
  rotate_rows(v, smem + seg * kSlotBytes, lane, f);
  mx_store<0>(f, row, t.rows, K, g, lane, codes, scales);
}

// An e2m1 code as the integer 2 c: 0 1 2 3 4 6 8 12 and their negatives.
__device__ __forceinline__ int e2m1_twice(uint32_t code) {
  const int m = (int)((0xC8643210u >> (4 * (code & 7))) & 15u);
  return code & 8 ? -m : m;
}

// Un-rotation.  A value is a multiple of 2^e / 2 up to 6 2^e, so while the scales
// of a group lie within 2^12 of one another every partial sum of its 256 values
// fits fp32's 24 bits and the transform is exact there; groups beyond that (or at
// the ends of the scales' range, or with a NaN) take the fp64 one, whose sums are
// rounded to fp32 before they are rounded to the type.  Blocks of zeros have no say.
template <bool kBF16>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t K, Units t,
                     uint16_t* __restrict__ V) {
  __shared__ __align__(16) char smem[kSegs * kSlotBytes];
  const int seg = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const uint32_t u = blockIdx.x * kSegs + seg;
  if (u >= t.total) return;
  uint32_t row, g;
  unit_of(t, u, row, g);
  const uint2 c = *reinterpret_cast<const uint2*>(codes + row * (K / 2) + g * 128 + 8 * lane);
  const uint32_t byte = scales[((int64_t)g * t.rows + row) * 8 + (lane >> 1)];
  const bool some = ((c.x | c.y) & 0x77777777u) != 0u;
  // largest scale and smallest (as the largest of 255 - byte) over the 16 lanes
  const uint32_t high = seg_max16_bits(some || byte == 255u ? byte : 0u);
  const uint32_t low = 255u - seg_max16_bits(some ? 255u - byte : 0u);
  char* slot = smem + seg * kSlotBytes;
  float f[16];
  if (high < 240u && low >= 8u && high <= low + 12u) {
    const float s = __uint_as_float((byte > 8u ? byte - 4u : 4u) << 23);   // 1/16 of it: the transform of +-1
    typedef float f2 __attribute__((ext_vector_type(2)));
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 1),
                       __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 3)};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[8 * j + 2 * i] = p[i][0], f[8 * j + 2 * i + 1] = p[i][1];
    }
    rotate_rows(f, slot, lane);
  } else {
    // 2^(byte - 127) / 2 (the codes are taken twice) / 16
    const double s = byte == 255u ? __longlong_as_double(0x7FF8000000000000ll)
                                  : __longlong_as_double((long long)(byte + 1023 - 127 - 5) << 52);
    double v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = (double)e2m1_twice((i < 8 ? c.x : c.y) >> (4 * (i & 7))) * s;
    rotate_rows(v, slot, lane, f);
  }
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    o[i] = kBF16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){f[2 * i], f[2 * i + 1]}, b2))
                 : pack_f16x2_rn(f[2 * i], f[2 * i + 1]);
  }
  uint4* dst = reinterpret_cast<uint4*>(V + row * K + g * kGroup + 16 * lane);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

dim3 grid_of(const Units& t) { return dim3((t.total + kSegs - 1) / kSegs); }

}  // namespace

hipError_t launch_mx_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* codes, uint8_t* scales,
                                      hipStream_t stream) {
  const Units t = units(N, K);
  hipLaunchKernelGGL(mx_quantize_weights_kernel, grid_of(t), dim3(256), 0, stream, W, K, t, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_act_quant(const void* X, bool bf16, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream) {
  const auto fn = bf16 ? &mx_act_quant_kernel<true> : &mx_act_quant_kernel<false>;
  int64_t resident = 0;
  if (const hipError_t e = resident_grid(reinterpret_cast<const void*>(fn), 256, 0, &resident); e != hipSuccess) return e;
  const Units t = units(M, K);
  const dim3 all = grid_of(t);
  hipLaunchKernelGGL(fn, all.x < resident ? all : dim3((unsigned)resident), dim3(256), 0, stream,
                     static_cast<const uint16_t*>(X), K, t, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* V,
                                bool bf16, hipStream_t stream) {
  const auto fn = bf16 ? &mx_dequantize_kernel<true> : &mx_dequantize_kernel<false>;
  const Units t = units(rows, K);
  hipLaunchKernelGGL(fn, grid_of(t), dim3(256), 0, stream, codes, scales, K, t, static_cast<uint16_t*>(V));
  return hipGetLastError();
}

}  // namespace convrot
