// The norms around the linears with outputs of 16 bits: the norm in front of one
// with its shift and scale, and the gated residual behind a block with the norm of
// the next (norm_quant.hip rotates and quantises them for the linear that follows).
//
// Mathematics.  h = residual_scale x + gate post(y) (or x), n = ((h - mu) r
// weight + bias)(1 + scale) + shift, in one pass: a row is held in registers
// from its load to its last output.  It is fp32.  The mean is taken first,
// then the sums of d = h - mu and of d^2; what the first says that mu is off stays
// apart, so that rows of one value give 0 and a mean far above the spread costs no
// digits.  Rows that fp32 does not hold are taken in fp64.
//
// Work split.  WAVES wavefronts own a row, each lane S units of 8 neighbouring
// elements (one 16-byte load).  One wavefront a row needs no barrier; four such
// rows share a workgroup.  Rows need no alignment: the loads are 16 bytes at any
// element, a last partial unit goes element by element.
//
// Bound and measured (us, one call after another in a graph, inputs in turn, bf16).
// 16384 rows of 2048 by memory: norm 24.5, residual with a norm of y and the next norm
// 52 (5.2 TB/s, as a large copy), h alone 33 (the last cache holds part of the inputs
// of the first and the third).  1024 rows 3.7 and 6.5, 3 rows 2.7 and 3.8: latency, the
// parameters' loads behind the sums one after another.

#include "norm_core.hpp"

namespace convrot {
namespace {

// Sum over the wavefront, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Sums over the row's wavefronts, in their order (b only where kTwo).  `part` is
// written by this sum alone until the next barrier has passed.
template <int WAVES, bool kTwo>
__device__ __forceinline__ void row_sums(float& a, float& b, float2* part) {
  a = wave_sum(a);
  if constexpr (kTwo) b = wave_sum(b);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    float2 s = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const float2 t = part[w];
      s.x += t.x;
      s.y += t.y;
    }
    a = s.x;
    b = s.y;
  }
}

// What the sums of a row's wavefronts pass through.
struct RowParts {
  float2 means[16], sums[16];
};

// A row in fp32, unit k's 8 elements in v[k] (0 past the row's end; `first(k)` is the
// unit's first element), to (v - mu) r.  The mean is mu + e: e, the mean of the
// differences, is what the rounding of mu left, and stays apart, since a mean far
// above the spread may lie between two fp32 numbers.  Rows that fp32 does not hold are
// taken in fp64: those whose squares leave its range, and those where e passes the
// spread itself (rows of one value among them, which then give 0).
template <int S, int WAVES, typename First>
__device__ __forceinline__ void normalise(float (&v)[S][8], First first, int kind, float eps, const NormArgs& a,
                                          RowParts& parts, double (*wide)[16]) {
  const int D = a.D;
  float mu = 0.0f, none = 0.0f, e = 0.0f, q = 0.0f;
  if (kind == kNormLayer) {
#pragma unroll
    for (int k = 0; k < S; ++k)
      mu += ((v[k][0] + v[k][1]) + (v[k][2] + v[k][3])) + ((v[k][4] + v[k][5]) + (v[k][6] + v[k][7]));
    row_sums<WAVES, false>(mu, none, parts.means);
    mu *= a.inv_d;
  }
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int left = D - first(k);
    float p[8], w = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[k][i] - mu;
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = i < left ? p[i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w = __fmaf_rn(p[i], p[i], w);
    q += w;
    if (kind == kNormLayer) e += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
  }
  row_sums<WAVES, true>(e, q, parts.sums);
  mu = as_fp32(mu);   // so that the differences are taken again, and do not hold registers next to v
  e *= a.inv_d;
  const float var = __fmaf_rn(-e, e, q * a.inv_d);
  // the same bits in every lane of the row's wavefronts; an infinity or a NaN fails too
  if (__builtin_expect(q <= 0x1p120f && var + eps >= 0x1p-90f && e * e <= var, 1)) {
    const float r = __builtin_amdgcn_rsqf(var + eps);   // within one ulp
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = ((v[k][i] - mu) - e) * r;
    return;
  }
  // rare: one element after the other, in few registers, so that the ordinary rows keep theirs
  double m = 0.0, z = 0.0;
  if (kind == kNormLayer) {
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m += (double)as_fp32(v[k][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    m = quotient(row_sum<WAVES>(m, wide[0]), (double)D, a.inv_wide);
  }
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = first(k) + i < D ? (double)as_fp32(v[k][i]) - m : 0.0;
      z = __fma_rn(d, d, z);
      __builtin_amdgcn_sched_barrier(0);
    }
  z = inverse_root(row_sum<WAVES>(z, wide[1]) * a.inv_wide + (double)eps);
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[k][i] = (float)(((double)v[k][i] - m) * z);
      __builtin_amdgcn_sched_barrier(0);
    }
}

// t = t weight + bias.
template <int S, typename First>
__device__ __forceinline__ void affine(float (&t)[S][8], First first, const NormDesc& n, int D) {
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int e0 = first(k);
    if (e0 >= D) continue;
    float p[8];
    if (n.weight) {
      load8<false>(n.weight, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] *= p[i];
    }
    if (n.bias) {
      load8<false>(n.bias, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] += p[i];
    }
  }
}

template <bool kBF16, int OUT, bool RES, int S, int WAVES>
__global__ void __launch_bounds__(WAVES <= 4 ? 256 : 64 * WAVES)
norm_kernel(NormArgs a) {
  __shared__ RowParts parts[2];
  __shared__ double wide[2][16];   // of both norms: a barrier of the second's sums lies between
  const int lane = threadIdx.x & 63, wave_id = threadIdx.x >> 6;
  const int wave = WAVES == 1 ? 0 : wave_id;
  const uint32_t row32 = WAVES == 1 ? blockIdx.x * (blockDim.x >> 6) + wave_id : blockIdx.x;
  if (row32 >= a.M) return;
  const uint32_t mrow32 = mod_row(a, row32);
  if (mrow32 >= a.mod_rows) return;       // of no sequence (negative ones too): the whole row's wavefronts leave
  const int64_t row = row32, mrow = mrow32;
  const int D = a.D;
  auto first = [&](int k) { return ((wave + WAVES * k) * 64 + lane) * 8; };
  auto widen8 = [](v8u raw, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = widen<kBF16>(raw[i]);
  };

  v8u xr[S];
#pragma unroll
  for (int k = 0; k < S; ++k) xr[k] = load8<false>(a.x + row * a.x_stride, first(k), D);
  float v[S][8];
  if constexpr (RES) {
    v8u yr[S];
#pragma unroll
    for (int k = 0; k < S; ++k) yr[k] = load8<false>(a.y + row * a.y_stride, first(k), D);
#pragma unroll
    for (int k = 0; k < S; ++k) widen8(yr[k], v[k]);
    if (a.post.kind != kNormNone) {
      normalise<S, WAVES>(v, first, a.post.kind, a.post.eps, a, parts[0], wide);
      affine<S>(v, first, a.post, D);
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int e0 = first(k), left = D - e0;
      if (a.gate && left > 0) {
        float p[8];
        load_mod<kBF16, false>(a.gate, mrow * a.gate_stride, a.mod_f32, e0, D, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= p[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = __fmaf_rn(a.residual_scale, widen<kBF16>(xr[k][i]), v[k][i]);
        v[k][i] = i < left ? h : 0.0f;
      }
      if (left > 0) store8<false>(a.h + row * D, e0, D, narrow<kBF16>(v[k]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < S; ++k) widen8(xr[k], v[k]);
  }
  if constexpr (OUT == kOutNone) return;

  normalise<S, WAVES>(v, first, a.norm.kind, a.norm.eps, a, parts[1], wide);
  affine<S>(v, first, a.norm, D);
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int e0 = first(k);
    if (e0 >= D) continue;
    float p[8];
    if (a.scale) {
      load_mod<kBF16, false>(a.scale, mrow * a.scale_stride, a.mod_f32, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = __fmaf_rn(v[k][i], p[i], v[k][i]);
    }
    if (a.shift) {
      load_mod<kBF16, false>(a.shift, mrow * a.shift_stride, a.mod_f32, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] += p[i];
    }
    store8<false>(static_cast<uint16_t*>(a.values) + row * D, e0, D, narrow<kBF16>(v[k]));
  }
}

template <bool kBF16, int OUT, bool RES, int S, int WAVES>
hipError_t launch(const NormArgs& a, hipStream_t stream) {
  const int rows = WAVES == 1 ? 4 : 1;
  hipLaunchKernelGGL((norm_kernel<kBF16, OUT, RES, S, WAVES>), dim3((a.M + rows - 1) / rows), dim3(64 * WAVES * rows),
                     0, stream, a);
  return hipGetLastError();
}

// Wavefronts a row and units a lane: two units where that still leaves 8 wavefronts
// a CU (16384 rows of 2048: norm 26.8 against 30.3 us, residual 55 against 58; 4000
// rows of 5000: norm 21 against 26, residual 41 against 43), else one, which is faster
// by latency (1024 rows of 1024: norm 4.4 against 4.9 us, residual 5.6 against 6.6).
// Four units a lane (residual, one wavefront a row of 2048) leave 3 wavefronts a
// SIMD: 74 us.  A grid has fewer than 2^32 threads in every case: with M D at most
// 2^35 the most are 2^35 / 2049 rows of 256, 2^35 / 4097 of 512 and 2^35 / 8193 of 1024.
template <bool kBF16, int OUT, bool RES>
hipError_t choose(const NormArgs& a, hipStream_t stream) {
  const int units = (a.D + 511) / 512;   // of a wavefront's lanes, over the row
  if (units <= 1) return launch<kBF16, OUT, RES, 1, 1>(a, stream);
  if ((int64_t)a.M * units > 4096) {
    if (units <= 2) return launch<kBF16, OUT, RES, 2, 1>(a, stream);
    if (units <= 4) return launch<kBF16, OUT, RES, 2, 2>(a, stream);
    if (units <= 8) return launch<kBF16, OUT, RES, 2, 4>(a, stream);
    if (units <= 16) return launch<kBF16, OUT, RES, 2, 8>(a, stream);
  }
  if (units <= 2) return launch<kBF16, OUT, RES, 1, 2>(a, stream);
  if (units <= 4) return launch<kBF16, OUT, RES, 1, 4>(a, stream);
  if (units <= 8) return launch<kBF16, OUT, RES, 1, 8>(a, stream);
  if (units <= 16) return launch<kBF16, OUT, RES, 1, 16>(a, stream);
  return launch<kBF16, OUT, RES, 2, 16>(a, stream);
}

template <bool kBF16>
hipError_t by_output(const NormArgs& a, NormOut out, hipStream_t stream) {
  if (out == kOutNone) return choose<kBF16, kOutNone, true>(a, stream);
  return a.y ? choose<kBF16, kOut16, true>(a, stream) : choose<kBF16, kOut16, false>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, NormOut out, hipStream_t stream) {
  if (out == kOutInt8 || out == kOutMx) return launch_norm_quant(a, bf16, out, stream);
  return bf16 ? by_output<true>(a, out, stream) : by_output<false>(a, out, stream);
}

}  // namespace convrot
