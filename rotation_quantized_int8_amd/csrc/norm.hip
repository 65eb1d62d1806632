// The norms around the linears: the norm in front of one with its shift and
// scale, and the gated residual behind a block with the norm of the next, to 16
// bits or rotated and quantised for the linear that follows.
//
// Mathematics.  h = residual_scale x + gate post(y) (or x), n = ((h - mu) r
// weight + bias)(1 + scale) + shift, in one pass: a row is held in registers
// from its load to its last output, its statistics are two sums over the lanes
// (the mean first, then the squares of the differences, so that nothing
// cancels).  All of it is fp64: gfx950 issues fp64 additions and fused
// multiply-adds at the rate of single fp32 ones, the rows are bound by memory,
// and so no square overflows and codes come out as those of the formula.
//
// Work split.  `waves` wavefronts own a row, each lane units of V neighbouring
// elements: 8 (one 16-byte load) for outputs of 16 bits, 16 (a row of the
// rotation's 16 x 16 view) for quantised ones, S units a lane.  One wavefront a
// row needs no barrier; four such rows share a workgroup.  Rows need no
// alignment: the loads are 16 bytes at any element, a last partial unit goes
// element by element.

#include "norm.hpp"

namespace convrot {
namespace {

typedef uint16_t v8u __attribute__((ext_vector_type(8)));
typedef v8u v8u_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

__device__ __forceinline__ double dpp_f64(double v, const int step) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  switch (step) {
    case 0: lo = __builtin_amdgcn_update_dpp(0, lo, 0xB1, 0xF, 0xF, true);
            hi = __builtin_amdgcn_update_dpp(0, hi, 0xB1, 0xF, 0xF, true); break;
    case 1: lo = __builtin_amdgcn_update_dpp(0, lo, 0x4E, 0xF, 0xF, true);
            hi = __builtin_amdgcn_update_dpp(0, hi, 0x4E, 0xF, 0xF, true); break;
    case 2: lo = __builtin_amdgcn_update_dpp(0, lo, 0x141, 0xF, 0xF, true);
            hi = __builtin_amdgcn_update_dpp(0, hi, 0x141, 0xF, 0xF, true); break;
    default: lo = __builtin_amdgcn_update_dpp(0, lo, 0x140, 0xF, 0xF, true);
             hi = __builtin_amdgcn_update_dpp(0, hi, 0x140, 0xF, 0xF, true); break;
  }
  return __longlong_as_double((long long)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo));
}

// Sum over the wavefront, the same bits in every lane.
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int s = 0; s < 4; ++s) v += dpp_f64(v, s);
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  v = __longlong_as_double((long long)((uint64_t)h[0] << 32 | l[0])) +
      __longlong_as_double((long long)((uint64_t)h[1] << 32 | l[1]));
  const uint64_t w = (uint64_t)__double_as_longlong(v);
  const auto l2 = __builtin_amdgcn_permlane32_swap((uint32_t)w, (uint32_t)w, false, false);
  const auto h2 = __builtin_amdgcn_permlane32_swap((uint32_t)(w >> 32), (uint32_t)(w >> 32), false, false);
  return __longlong_as_double((long long)((uint64_t)h2[0] << 32 | l2[0])) +
         __longlong_as_double((long long)((uint64_t)h2[1] << 32 | l2[1]));
}

// Sum over the row's wavefronts, in their order; `part` is used by this sum
// alone (one of the kernel's, so that no barrier has to free it).
__device__ __forceinline__ double row_sum(double v, int waves, double* part) {
  v = wave_sum_f64(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < waves; ++w) v += part[w];
  return v;
}

template <bool kBF16>
__device__ __forceinline__ double widen(uint16_t b) {
  return kBF16 ? (double)bf16_to_f32(b) : (double)__half2float(__ushort_as_half(b));
}
template <bool kBF16>
__device__ __forceinline__ uint16_t narrow(double v) {
  const float f = (float)v;
  return kBF16 ? f32_to_bf16_rn(f) : __half_as_ushort(__float2half_rn(as_fp32(f)));
}

// 8 neighbouring elements from e0 of a 16-bit row of D (zeros past its end).
__device__ __forceinline__ v8u load8(const uint16_t* row, int e0, int D) {
  if (e0 + 8 <= D) return *reinterpret_cast<const v8u_any*>(row + e0);
  v8u v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e0 + i < D) v[i] = row[e0 + i];
  return v;
}
__device__ __forceinline__ void load8(const float* row, int e0, int D, float (&f)[8]) {
  if (e0 + 8 <= D) {
    const v4f a = *reinterpret_cast<const v4f_any*>(row + e0), b = *reinterpret_cast<const v4f_any*>(row + e0 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e0 + i < D ? row[e0 + i] : 0.0f;
  }
}
// The same of a modulation's row.
template <bool kBF16>
__device__ __forceinline__ void load_mod(const void* base, int64_t at, int f32, int e0, int D, float (&f)[8]) {
  if (f32) {
    load8(static_cast<const float*>(base) + at, e0, D, f);
  } else {
    const v8u v = load8(static_cast<const uint16_t*>(base) + at, e0, D);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)widen<kBF16>(v[i]);
  }
}
__device__ __forceinline__ void store8(uint16_t* row, int e0, int D, v8u v) {
  if (e0 + 8 <= D) {
    *reinterpret_cast<v8u_any*>(row + e0) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i < D) row[e0 + i] = v[i];
  }
}

// mu and r of the row that the lanes hold in v (zeros past its end).
template <int V, int S>
__device__ __forceinline__ void statistics(const double (&v)[S][V], int kind, double eps, int D, int waves,
                                           int wave, int lane, double (*part)[16], double& mu, double& r) {
  mu = 0.0;
  if (kind == kNormLayer) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[k][i];
    mu = row_sum(s, waves, part[0]) / D;
  }
  double q = 0.0;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int e0 = ((wave + waves * k) * 64 + lane) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double d = e0 + i < D ? v[k][i] - mu : 0.0;
      q = __fma_rn(d, d, q);
    }
  }
  r = 1.0 / sqrt(row_sum(q, waves, part[1]) / D + eps);
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

template <bool kBF16, int OUT, bool RES, int S>
__global__ void __launch_bounds__(1024)
norm_kernel(NormArgs a, int waves) {
  constexpr int V = OUT == kOutInt8 || OUT == kOutMx ? 16 : 8;
  constexpr bool kTurn = V == 16;
  extern __shared__ __align__(16) char slots[];     // quantised: a slot for each group in work
  __shared__ double part[4][16];
  __shared__ uint32_t top[16];
  const int lane = threadIdx.x & 63, wave_id = threadIdx.x >> 6;
  const int wave = waves == 1 ? 0 : wave_id;
  const int64_t row = waves == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + wave_id : blockIdx.x;
  if (row >= a.M) return;
  const int64_t mrow = a.index ? a.index[row] : row / a.each;
  if (mrow < 0 || mrow >= a.mod_rows) return;       // of no sequence: the whole row's wavefronts leave
  const int D = a.D;
  auto first = [&](int k) { return ((wave + waves * k) * 64 + lane) * V; };

  double v[S][V];
  {
    const uint16_t* xr = a.x + row * a.x_stride;
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < V; c += 8) {
        const v8u t = load8(xr, first(k) + c, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][c + i] = widen<kBF16>(t[i]);
      }
  }
  if constexpr (RES) {
    double y[S][V];
    const uint16_t* yr = a.y + row * a.y_stride;
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < V; c += 8) {
        const v8u t = load8(yr, first(k) + c, D);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[k][c + i] = widen<kBF16>(t[i]);
      }
    double mu = 0.0, r = 1.0;
    if (a.post.kind != kNormNone)
      statistics<V, S>(y, a.post.kind, (double)a.post.eps, D, waves, wave, lane, &part[0], mu, r);
    uint16_t* hr = a.h + row * D;
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < V; c += 8) {
        const int e0 = first(k) + c;
        if (e0 >= D) continue;
        float w[8] = {1, 1, 1, 1, 1, 1, 1, 1}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8] = {1, 1, 1, 1, 1, 1, 1, 1};
        if (a.post.weight) load8(a.post.weight, e0, D, w);
        if (a.post.bias) load8(a.post.bias, e0, D, b);
        if (a.gate) load_mod<kBF16>(a.gate, mrow * a.gate_stride, a.mod_f32, e0, D, g);
        v8u o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double t = __fma_rn((y[k][c + i] - mu) * r, (double)w[i], (double)b[i]);
          const double h = __fma_rn((double)g[i], t, a.residual_scale * v[k][c + i]);
          v[k][c + i] = e0 + i < D ? h : 0.0;
          o[i] = narrow<kBF16>(h);
        }
        store8(hr, e0, D, o);
      }
  }
  if constexpr (OUT == kOutNone) return;

  double mu, r;
  statistics<V, S>(v, a.norm.kind, (double)a.norm.eps, D, waves, wave, lane, &part[2], mu, r);
  float f[kTurn ? S : 1][16];
  const int seg = (int)threadIdx.x >> 4, sl = lane & 15;
#pragma unroll
  for (int k = 0; k < S; ++k) {
#pragma unroll
    for (int c = 0; c < V; c += 8) {
      const int e0 = first(k) + c;
      if (e0 >= D) continue;
      float w[8] = {1, 1, 1, 1, 1, 1, 1, 1}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      float sc[8] = {0, 0, 0, 0, 0, 0, 0, 0}, sh[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (a.norm.weight) load8(a.norm.weight, e0, D, w);
      if (a.norm.bias) load8(a.norm.bias, e0, D, b);
      if (a.scale) load_mod<kBF16>(a.scale, mrow * a.scale_stride, a.mod_f32, e0, D, sc);
      if (a.shift) load_mod<kBF16>(a.shift, mrow * a.shift_stride, a.mod_f32, e0, D, sh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double t = __fma_rn((v[k][c + i] - mu) * r, (double)w[i], (double)b[i]);
        v[k][c + i] = __fma_rn(t, 1.0 + (double)sc[i], (double)sh[i]);
      }
      if constexpr (!kTurn) {
        v8u o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = narrow<kBF16>(v[k][c + i]);
        store8(static_cast<uint16_t*>(a.values) + row * D, e0, D, o);
      }
    }
    if constexpr (kTurn) {
      // D is a multiple of 256, so the 16 lanes of a group are all inside or all outside
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[k][i] = __fma_rn(v[k][i], 0.0625, 0.0);   // a zero becomes +0
        f[k][i] = 0.0f;
      }
      if (first(k) < D) rotate_rows(v[k], slots + seg * kSlotBytes, sl, f[k]);
    }
  }
  if constexpr (OUT == kOutMx) {
#pragma unroll
    for (int k = 0; k < S; ++k)
      if (first(k) < D)
        mx_store<0>(f[k], row, a.M, D, first(k) / kGroup, sl, static_cast<uint8_t*>(a.values),
                    static_cast<uint8_t*>(a.scales));
  }
  if constexpr (OUT == kOutInt8) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[k][i]) & 0x7FFFFFFFu);
    m = seg_max16_bits(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (waves > 1) {
      if (lane == 0) top[wave] = m;
      __syncthreads();
      m = top[0];
      for (int w = 1; w < waves; ++w) m = max(m, top[w]);
    }
    const bool finite = m < 0x7F800000u;
    const float s = finite ? __uint_as_float(m) / 127.0f : __uint_as_float(0x7FC00000u);
    if (wave == 0 && lane == 0) static_cast<float*>(a.scales)[row] = s;
#pragma unroll
    for (int k = 0; k < S; ++k)
      if (first(k) < D)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.values) + row * D + first(k)) =
            finite ? codes16(f[k], s) : make_uint4(0, 0, 0, 0);
  }
}

template <bool kBF16, int OUT, bool RES, int S>
hipError_t launch(const NormArgs& a, int waves, hipStream_t stream) {
  constexpr bool kTurn = OUT == kOutInt8 || OUT == kOutMx;
  const int rows = waves == 1 ? 4 : 1, threads = 64 * waves * rows;
  const size_t lds = kTurn ? (size_t)threads / 16 * kSlotBytes : 0;
  const auto fn = &norm_kernel<kBF16, OUT, RES, S>;
  if (const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(fn), lds); e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((unsigned)((a.M + rows - 1) / rows)), dim3(threads), lds, stream, a, waves);
  return hipGetLastError();
}

// Wavefronts a row and units a lane: one wavefront with up to 32 elements a
// lane (no barrier), more for wider rows.
template <bool kBF16, int OUT, bool RES>
hipError_t choose(const NormArgs& a, hipStream_t stream) {
  constexpr int V = OUT == kOutInt8 || OUT == kOutMx ? 16 : 8, kMost = 32 / V;
  const int units = (a.D + 64 * V - 1) / (64 * V);   // of a wavefront's lanes, over the row
  int waves = 1;
  while (waves * kMost < units) waves *= 2;
  const int s = (units + waves - 1) / waves;
  if (s == 1) return launch<kBF16, OUT, RES, 1>(a, waves, stream);
  if (s == 2 || kMost == 2) return launch<kBF16, OUT, RES, 2>(a, waves, stream);
  return launch<kBF16, OUT, RES, kMost>(a, waves, stream);
}

template <bool kBF16>
hipError_t by_output(const NormArgs& a, NormOut out, hipStream_t stream) {
  switch (out) {
    case kOutNone: return choose<kBF16, kOutNone, true>(a, stream);
    case kOut16: return a.y ? choose<kBF16, kOut16, true>(a, stream) : choose<kBF16, kOut16, false>(a, stream);
    case kOutInt8: return a.y ? choose<kBF16, kOutInt8, true>(a, stream) : choose<kBF16, kOutInt8, false>(a, stream);
    default: return a.y ? choose<kBF16, kOutMx, true>(a, stream) : choose<kBF16, kOutMx, false>(a, stream);
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, NormOut out, hipStream_t stream) {
  return bf16 ? by_output<true>(a, out, stream) : by_output<false>(a, out, stream);
}

}  // namespace convrot
