// The norms around the linears with outputs of 16 bits: the norm in front of one
// with its shift and scale, and the gated residual behind a block with the norm of
// the next (norm_quant.hip rotates and quantises them for the linear that follows).
//
// Mathematics.  h = residual_scale x + gate post(y) (or x), n = ((h - mu) r
// weight + bias)(1 + scale) + shift, in one pass: a row is held in registers
// from its load to its last output.  All of it is fp32.  The mean is taken first,
// then the sums of d = h - mu and of d^2, whose first takes out what the rounding
// of mu left, so that rows of one value give 0 and a mean far above the spread
// costs no digits.  A row whose squares leave fp32's range is taken times a power
// of two instead.
//
// Work split.  WAVES wavefronts own a row, each lane S units of 8 neighbouring
// elements (one 16-byte load).  One wavefront a row needs no barrier; four such
// rows share a workgroup.  Rows need no alignment: the loads are 16 bytes at any
// element, a last partial unit goes element by element.
//
// Bound and measured (us on the GPU, inputs in turn, 16384 rows of 2048 in bf16):
// memory: norm 27 (5.0 TB/s), residual with a norm of y and the next norm 54 (5.0
// TB/s; a large copy reaches 5.1).

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

constexpr float kSmall = 0x1p-90f, kUp = 0x1p96f;

// A row in fp32, element i of unit k as at(k, i) (0 past the row's
// end; `first(k)` is the unit's first element), to its mu and r: t = (at - mu) r.
// kRange: the row may leave the range of fp32's squares (fp16 ones do not).  Then
// `scale_by` multiplies it by a power of two, which t does not feel: a row whose
// squares pass fp32 is taken 2^-96 times, one whose squares vanish next to a
// vanishing eps 2^96 times.  (With a mean beyond 1 such a row has no spread at all:
// its differences would be at least the spacing of its values.)
template <int S, int WAVES, bool kRange, typename At, typename First, typename ScaleBy>
__device__ __forceinline__ void statistics(At at, First first, ScaleBy scale_by, int kind, float eps, int D,
                                           float inv, float2 (*part)[16], float& mu, float& r) {
  for (int round = 0;; ++round) {
    mu = 0.0f;
    if (kind == kNormLayer) {
      float s = 0.0f, none = 0.0f;
#pragma unroll
      for (int k = 0; k < S; ++k) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = at(k, i);
        s += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      }
      row_sums<WAVES, false>(s, none, part[0]);
      mu = s * inv;
    }
    float e = 0.0f, q = 0.0f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int left = D - first(k);
      float p[8], w = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = at(k, i) - mu;
      if (left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = i < left ? p[i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) w = __fmaf_rn(p[i], p[i], w);
      q += w;
      if (kind == kNormLayer) e += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    }
    row_sums<WAVES, true>(e, q, part[1 + round]);
    e *= inv;
    const float var = fmaxf(__fmaf_rn(-e, e, q * inv), 0.0f) + eps;
    mu += e;
    r = __builtin_amdgcn_rsqf(var);   // within one ulp
    if (!kRange || round || (q <= 0x1p120f && (var >= kSmall || fabsf(mu) > 1.0f))) return;
    const float by = q <= 0x1p120f ? kUp : 1.0f / kUp;
    scale_by(by);
    if (eps > 0.0f) eps = fmaxf(eps * by * by, 0x1p-126f);   // still above 0: a row of one value gives 0
  }
}

template <bool kBF16, int OUT, bool RES, int S, int WAVES>
__global__ void __launch_bounds__(WAVES <= 4 ? 256 : 64 * WAVES)
norm_kernel(NormArgs a) {
  __shared__ float2 part[6][16];
  const int lane = threadIdx.x & 63, wave_id = threadIdx.x >> 6;
  const int wave = WAVES == 1 ? 0 : wave_id;
  const uint32_t row32 = WAVES == 1 ? blockIdx.x * (blockDim.x >> 6) + wave_id : blockIdx.x;
  if (row32 >= a.M) return;
  const uint32_t mrow32 = mod_row(a, row32);
  if (mrow32 >= a.mod_rows) return;       // of no sequence (negative ones too): the whole row's wavefronts leave
  const int64_t row = row32, mrow = mrow32;
  const int D = a.D;
  auto first = [&](int k) { return ((wave + WAVES * k) * 64 + lane) * 8; };

  v8u xr[S];
#pragma unroll
  for (int k = 0; k < S; ++k) xr[k] = load8<false>(a.x + row * a.x_stride, first(k), D);
  auto rescale = [&](v8u (&raw)[S], float by) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = widen<kBF16>(raw[k][i]) * by;
      raw[k] = narrow<kBF16>(p);
    }
  };
  float h[RES ? S : 1][8];   // the residual form's rows in fp32; x itself is widened where it is read
  if constexpr (RES) {
    v8u yr[S];
#pragma unroll
    for (int k = 0; k < S; ++k) yr[k] = load8<false>(a.y + row * a.y_stride, first(k), D);
    float mu = 0.0f, r = 1.0f;
    if (a.post.kind != kNormNone)
      statistics<S, WAVES, kBF16>([&](int k, int i) { return widen<kBF16>(yr[k][i]); }, first,
                                  [&](float by) { rescale(yr, by); }, a.post.kind, a.post.eps, D, a.inv_d, &part[0],
                                  mu, r);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int e0 = first(k);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = 0.0f;
      if (e0 >= D) continue;
      float t[8], p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = widen<kBF16>(yr[k][i]);
      if (a.post.kind != kNormNone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = (t[i] - mu) * r;
        if (a.post.weight) {
          load8<false>(a.post.weight, e0, D, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] *= p[i];
        }
        if (a.post.bias) {
          load8<false>(a.post.bias, e0, D, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] += p[i];
        }
      }
      if (a.gate) {
        load_mod<kBF16, false>(a.gate, mrow * a.gate_stride, a.mod_f32, e0, D, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= p[i];
      }
      const int left = D - e0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __fmaf_rn(a.residual_scale, widen<kBF16>(xr[k][i]), t[i]);
        h[k][i] = i < left ? v : 0.0f;
      }
      store8<false>(a.h + row * D, e0, D, narrow<kBF16>(h[k]));
    }
  }
  if constexpr (OUT == kOutNone) return;
  auto at = [&](int k, int i) {
    if constexpr (RES) return h[k][i];
    else return widen<kBF16>(xr[k][i]);
  };

  float mu, r;
  statistics<S, WAVES, kBF16 || RES>(
      at, first,
      [&](float by) {
        if constexpr (RES) {
#pragma unroll
          for (int k = 0; k < S; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) h[k][i] *= by;
        } else {
          rescale(xr, by);
        }
      },
      a.norm.kind, a.norm.eps, D, a.inv_d, &part[3], mu, r);
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int e0 = first(k);
    if (e0 >= D) continue;
    float t[8], p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = (at(k, i) - mu) * r;
    if (a.norm.weight) {
      load8<false>(a.norm.weight, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] *= p[i];
    }
    if (a.norm.bias) {
      load8<false>(a.norm.bias, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] += p[i];
    }
    if (a.scale) {
      load_mod<kBF16, false>(a.scale, mrow * a.scale_stride, a.mod_f32, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = __fmaf_rn(t[i], p[i], t[i]);
    }
    if (a.shift) {
      load_mod<kBF16, false>(a.shift, mrow * a.shift_stride, a.mod_f32, e0, D, p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] += p[i];
    }
    store8<false>(static_cast<uint16_t*>(a.values) + row * D, e0, D, narrow<kBF16>(t));
  }
}

template <bool kBF16, int OUT, bool RES, int S, int WAVES>
hipError_t launch(const NormArgs& a, hipStream_t stream) {
  const int rows = WAVES == 1 ? 4 : 1;
  hipLaunchKernelGGL((norm_kernel<kBF16, OUT, RES, S, WAVES>), dim3((a.M + rows - 1) / rows), dim3(64 * WAVES * rows),
                     0, stream, a);
  return hipGetLastError();
}

// Wavefronts a row and units a lane: two units where that still leaves 16 wavefronts
// a CU (16384 rows of 2048: norm 26.8 against 30.3 us, residual 55 against 58), else
// one, which is faster by latency (1024 rows of 1024: norm 4.4 against 4.9 us,
// residual 5.6 against 6.6).  Four units a lane (residual, one wavefront a row of
// 2048) leave 3 wavefronts a SIMD: 74 us.
template <bool kBF16, int OUT, bool RES>
hipError_t choose(const NormArgs& a, hipStream_t stream) {
  const int units = (a.D + 511) / 512;   // of a wavefront's lanes, over the row
  if (units <= 1) return launch<kBF16, OUT, RES, 1, 1>(a, stream);
  if ((int64_t)a.M * units > 4096) {
    if (units <= 2) return launch<kBF16, OUT, RES, 2, 1>(a, stream);
    if (units <= 4) return launch<kBF16, OUT, RES, 2, 2>(a, stream);
    if (units <= 8) return launch<kBF16, OUT, RES, 2, 4>(a, stream);
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
