// The norms around the linears, rotated and quantised for the linear that follows:
// the norm in front of one with its shift and scale, and the gated residual behind a
// block with the norm of the next, to int8 or to microscaled 4-bit floating point.
//
// Mathematics.  h = residual_scale x + gate post(y) (or x), n = ((h - mu) r
// weight + bias)(1 + scale) + shift, u = fp32(n H), in one pass.  A code is found by
// comparing u with borders, so an error before it shows as a whole step where u lies
// next to one: everything up to u is fp64, as in the other quantisers, and codes and
// scales are the formula's (in fp32 one code in 10^5 and half of the int8 scales
// were not).  The mean first, then the sum of the squares of h - mu; rows of one
// value give 0.  fp64 holds the squares of every row.
//
// Work split.  WAVES wavefronts own a row, each lane 16 neighbouring elements: a row
// of the rotation's 16 x 16 view, 16 lanes to a group.  One wavefront a row needs no
// barrier; four such rows share a workgroup.
//
// Bound and measured (us, one call after another in a graph, inputs in turn, bf16 rows
// of 2048, modulated; a call traced alone takes 1 to 4 more): 16384 rows to 4 bits 43
// (fp32: 26), to int8 45 (37), the residual form 70 and 69 (53 and 61): the vector
// unit, some 38 instructions an element of 4 to 5 cycles (an fp32 addition takes 2.8),
// at the 4 wavefronts a SIMD that the slots leave.  1024 rows 4.7 and 5.9 (4.3 and
// 6.0), residual 6.8 and 8.3; 3 rows 3.6 and 4.1, residual 4.6 and 5.2: latency of a
// row's chain (load, two sums, modulation, rotation).

#include "norm_core.hpp"

namespace convrot {
namespace {

template <int WAVES>
__device__ __forceinline__ void row_sums(double& a, double& b, double2* part) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_double2(a, b);
    __syncthreads();
    double2 s = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      s.x += part[w].x;
      s.y += part[w].y;
    }
    a = s.x;
    b = s.y;
  }
}

// The lane's 16 elements of a row (0 past its end) to v - mu, with the row's r; inv
// is 1 / D.  kRounded: values of more than the rows' few bits, whose sum may round:
// the mean's error, e, is taken out too, so that equal values end at 0.
template <int WAVES, bool kRounded>
__device__ __forceinline__ double statistics(double (&v)[16], bool inside, int kind, float eps, int D, double inv,
                                             double* mean_part, double2* part) {
  if (kind == kNormLayer) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 16; i += 4) s += (v[i] + v[i + 1]) + (v[i + 2] + v[i + 3]);
    s = row_sum<WAVES>(s, mean_part);
    const double mu = quotient(s, (double)D, inv);
    if (inside) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] -= mu;
    }
  }
  double q = 0.0, var;
#pragma unroll
  for (int i = 0; i < 16; ++i) q = __fma_rn(v[i], v[i], q);
  if (kRounded && kind == kNormLayer) {
    double e = 0.0;
#pragma unroll
    for (int i = 0; i < 16; i += 4) e += (v[i] + v[i + 1]) + (v[i + 2] + v[i + 3]);
    row_sums<WAVES>(e, q, part);
    e = quotient(e, (double)D, inv);
    var = __fma_rn(-e, e, q * inv);
    var = var < 0.0 ? 0.0 : var;   // a NaN stays
    if (inside) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] -= e;
    }
  } else {
    var = row_sum<WAVES>(q, reinterpret_cast<double*>(part)) * inv;
  }
  return inverse_root(var + (double)eps);
}

template <bool kBF16>
__device__ __forceinline__ void widen16(v8u a, v8u b, double (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = in16_to_f64<kBF16>(a[i]);
    v[8 + i] = in16_to_f64<kBF16>(b[i]);
  }
}
// 16 elements from e0 of a parameter [D], or of a modulation's row that begins at element `at`.
__device__ __forceinline__ void load16(const float* p, int e0, int D, double (&f)[16]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float t[8];
    load8<true>(p, e0 + 8 * c, D, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[8 * c + i] = (double)t[i];
  }
}
template <bool kBF16>
__device__ __forceinline__ void load_mod16(const void* base, int64_t at, int f32, int e0, int D, double (&f)[16]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float t[8];
    load_mod<kBF16, true>(base, at, f32, e0 + 8 * c, D, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[8 * c + i] = (double)t[i];
  }
}
// t = t weight + unit bias.
__device__ __forceinline__ void affine16(const NormDesc& n, int e0, int D, double unit, double (&t)[16]) {
  double p[16];
  if (n.weight) {
    load16(n.weight, e0, D, p);
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] *= p[i];
  }
  if (n.bias) {
    load16(n.bias, e0, D, p);
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = __fma_rn(p[i], unit, t[i]);
  }
}

// int8 codes of 16 values with the row's scale s > 0.  quantize16 multiplies
// by the reciprocal of s, which a very small s does not have in fp32's normal
// range: there the quotients are IEEE divisions, clamped since s itself is
// rounded coarsely.
__device__ __forceinline__ uint4 codes16(const float (&f)[16], float s) {
  if (s >= 0x1p-100f) return quantize16(f, s);
  uint32_t w[4] = {0, 0, 0, 0};
  if (s > 0.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i >> 2] |= ((uint32_t)(int)fminf(fmaxf(rintf(f[i] / s), -127.0f), 127.0f) & 255u) << (8 * (i & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr double kSixteenth = 0.0625;

template <bool kBF16, int OUT, bool RES, int WAVES>
__global__ void __launch_bounds__(WAVES <= 4 ? 256 : 64 * WAVES)
norm_quant_kernel(NormArgs a) {
  extern __shared__ __align__(16) char slots[];     // a slot for each group in work
  __shared__ double means[2][16];
  __shared__ double2 part[2][16];
  __shared__ uint32_t top[16];
  const int lane = threadIdx.x & 63, wave_id = threadIdx.x >> 6;
  const int wave = WAVES == 1 ? 0 : wave_id;
  // 4-bit scales of neighbouring rows share a line: each XCD (workgroup number mod 8) takes rows side by side, so
  // that its L2 puts the line together
  uint32_t block = blockIdx.x;
  if (OUT == kOutMx && (gridDim.x & 7) == 0) block = (block & 7) * (gridDim.x >> 3) + (block >> 3);
  const uint32_t row32 = WAVES == 1 ? block * (blockDim.x >> 6) + wave_id : block;
  if (row32 >= a.M) return;
  const uint32_t mrow32 = mod_row(a, row32);
  if (mrow32 >= a.mod_rows) return;       // of no sequence: the whole row's wavefronts leave
  const int64_t row = row32, mrow = mrow32;
  const int D = a.D, e0 = (wave * 64 + lane) * 16;
  const bool inside = e0 < D;             // D is a multiple of 256: of a group's 16 lanes all are inside or none

  const v8u x0 = load8<true>(a.x + row * a.x_stride, e0, D), x1 = load8<true>(a.x + row * a.x_stride, e0 + 8, D);
  double v[16];
  if constexpr (RES) {
    const v8u y0 = load8<true>(a.y + row * a.y_stride, e0, D), y1 = load8<true>(a.y + row * a.y_stride, e0 + 8, D);
    double t[16];
    widen16<kBF16>(y0, y1, t);
    if (a.post.kind != kNormNone) {
      const double r = statistics<WAVES, false>(t, inside, a.post.kind, a.post.eps, D, a.inv_wide, means[0], part[0]);
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] *= r;
      if (inside) affine16(a.post, e0, D, 1.0, t);
    }
    widen16<kBF16>(x0, x1, v);
    if (inside) {
      if (a.gate) {
        double p[16];
        load_mod16<kBF16>(a.gate, mrow * a.gate_stride, a.mod_f32, e0, D, p);
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] *= p[i];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[8 * c + i] = __fma_rn((double)a.residual_scale, v[8 * c + i], t[8 * c + i]);
          f[i] = (float)v[8 * c + i];
        }
        store8<true>(a.h + row * D, e0 + 8 * c, D, narrow<kBF16>(f));
      }
    }
  } else {
    widen16<kBF16>(x0, x1, v);
  }

  // n / 16 from here on: the rotation is that of +-1
  const double r =
      kSixteenth * statistics<WAVES, RES>(v, inside, a.norm.kind, a.norm.eps, D, a.inv_wide, means[1], part[1]);
  float f[16];   // u
  if (inside) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= r;
    affine16(a.norm, e0, D, kSixteenth, v);
    double p[16];
    if (a.scale) {
      load_mod16<kBF16>(a.scale, mrow * a.scale_stride, a.mod_f32, e0, D, p);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __fma_rn(v[i], p[i], v[i]);
    }
    if (a.shift) {
      load_mod16<kBF16>(a.shift, mrow * a.shift_stride, a.mod_f32, e0, D, p);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __fma_rn(p[i], kSixteenth, v[i]);
    }
    v[0] += 0.0;   // no -0: a sum of 0 is +0 (each has a difference of two terms or this one)
    const int sl = lane & 15;
    rotate_rows(v, slots + (threadIdx.x >> 4) * kSlotBytes, sl, f);
    if constexpr (OUT == kOutMx)
      mx_store<0>(f, row, a.M, D, e0 / kGroup, sl, static_cast<uint8_t*>(a.values), static_cast<uint8_t*>(a.scales));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 0.0f;
  }
  if constexpr (OUT == kOutInt8) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    m = seg_max16_bits(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (WAVES > 1) {
      if (lane == 0) top[wave] = m;
      __syncthreads();
      m = top[0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) m = max(m, top[w]);
    }
    const bool finite = m < 0x7F800000u;
    const float s = finite ? __uint_as_float(m) / 127.0f : __uint_as_float(0x7FC00000u);
    if (wave == 0 && lane == 0) static_cast<float*>(a.scales)[row] = s;
    if (inside)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.values) + row * D + e0) =
          finite ? codes16(f, s) : make_uint4(0, 0, 0, 0);
  }
}

template <bool kBF16, int OUT, bool RES, int WAVES>
hipError_t launch(const NormArgs& a, hipStream_t stream) {
  const int rows = WAVES == 1 ? 4 : 1, threads = 64 * WAVES * rows;
  const size_t lds = (size_t)threads / 16 * kSlotBytes;
  const auto fn = &norm_quant_kernel<kBF16, OUT, RES, WAVES>;
  if (const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(fn), lds); e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((a.M + rows - 1) / rows), dim3(threads), lds, stream, a);
  return hipGetLastError();
}

// Wavefronts a row: one unit of 16 elements a lane.  A grid has fewer than 2^32
// threads in every case, as those of norm.hip.
template <bool kBF16, int OUT, bool RES>
hipError_t choose(const NormArgs& a, hipStream_t stream) {
  const int units = (a.D + 1023) / 1024;
  if (units <= 1) return launch<kBF16, OUT, RES, 1>(a, stream);
  if (units <= 2) return launch<kBF16, OUT, RES, 2>(a, stream);
  if (units <= 4) return launch<kBF16, OUT, RES, 4>(a, stream);
  if (units <= 8) return launch<kBF16, OUT, RES, 8>(a, stream);
  return launch<kBF16, OUT, RES, 16>(a, stream);
}

template <bool kBF16, int OUT>
hipError_t by_input(const NormArgs& a, hipStream_t stream) {
  return a.y ? choose<kBF16, OUT, true>(a, stream) : choose<kBF16, OUT, false>(a, stream);
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, bool bf16, NormOut out, hipStream_t stream) {
  if (out == kOutInt8) return bf16 ? by_input<true, kOutInt8>(a, stream) : by_input<false, kOutInt8>(a, stream);
  return bf16 ? by_input<true, kOutMx>(a, stream) : by_input<false, kOutMx>(a, stream);
}

}  // namespace convrot
