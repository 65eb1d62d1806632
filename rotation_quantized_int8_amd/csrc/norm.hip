// The norms around the linears: the norm in front of one with its shift and
// scale, and the gated residual behind a block with the norm of the next, to 16
// bits or rotated and quantised for the linear that follows.
//
// Mathematics.  h = residual_scale x + gate post(y) (or x), n = ((h - mu) r
// weight + bias)(1 + scale) + shift, in one pass: a row is held in registers
// from its load to its last output.  All of it is fp32 (fp64 conversions issue at
// a quarter of the rate: the same kernel in fp64 took 49 instead of 33 us for
// 16384 x 2048 to 4 bits).  The mean is taken first, then the sums of d = h - mu
// and of d^2, whose first takes out what the rounding of mu left, so that rows of
// one value give 0 and a mean far above the spread costs no digits.  A row whose
// squares leave fp32's range is taken times a power of two instead.
//
// Work split.  WAVES wavefronts own a row, each lane S units of V neighbouring
// elements: 8 (one 16-byte load) for outputs of 16 bits, 16 (a row of the
// rotation's 16 x 16 view) for quantised ones.  One wavefront a row needs no
// barrier; four such rows share a workgroup.  Rows need no alignment: the loads
// are 16 bytes at any element, a last partial unit goes element by element.
//
// Bound and measured (us on the GPU, inputs in turn, 16384 rows of 2048 in bf16):
// 16-bit outputs by memory: norm 27 (5.0 TB/s), residual with a norm of y and the
// next norm 54 (5.0 TB/s; a large copy reaches 5.1).  Quantised ones by the vector
// unit (80 % busy with some 30 instructions an element, a third of them the rotation
// and the codes): to 4 bits 29 (2.9 TB/s; 30.2 with the rows widened where they are
// read).  1024 rows of 2048 to int8 8.2, 3 rows of the residual form to 4 bits 4.7:
// latency of a row's chain (load, two sums, modulation, rotation).

#include "norm.hpp"

namespace convrot {
namespace {

typedef uint16_t v8u __attribute__((ext_vector_type(8)));
typedef v8u v8u_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

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

constexpr float kSmall = 0x1p-90f, kUp = 0x1p96f;

// A row in fp32, element i of chunk c of unit k as at(k, c, i) (0 past the row's
// end; `first(k)` is the unit's first element), to its mu and r: t = (at - mu) r.
// kRange: the row may leave the range of fp32's squares (fp16 ones do not).  Then
// `scale_by` multiplies it by a power of two, which t does not feel: a row whose
// squares pass fp32 is taken 2^-96 times, one whose squares vanish next to a
// vanishing eps 2^96 times.  (With a mean beyond 1 such a row has no spread at all:
// its differences would be at least the spacing of its values.)
template <int V, int S, int WAVES, bool kRange, typename At, typename First, typename ScaleBy>
__device__ __forceinline__ void statistics(At at, First first, ScaleBy scale_by, int kind, float eps, int D,
                                           float inv, float2 (*part)[16], float& mu, float& r) {
  for (int round = 0;; ++round) {
    mu = 0.0f;
    if (kind == kNormLayer) {
      float s = 0.0f, none = 0.0f;
#pragma unroll
      for (int k = 0; k < S; ++k)
#pragma unroll
        for (int c = 0; c < V / 8; ++c) {
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = at(k, c, i);
          s += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        }
      row_sums<WAVES, false>(s, none, part[0]);
      mu = s * inv;
    }
    float e = 0.0f, q = 0.0f;
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < V / 8; ++c) {
        const int left = D - first(k) - 8 * c;
        if (V == 16 && left <= 0) continue;   // quantised rows: whole chunks
        float p[8], w = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = at(k, c, i) - mu;
        if (V == 8 && left < 8) {
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

template <bool kBF16, int OUT, bool RES, int S, int WAVES>
__global__ void __launch_bounds__(WAVES <= 4 ? 256 : 64 * WAVES)
norm_kernel(NormArgs a) {
  constexpr int V = OUT == kOutInt8 || OUT == kOutMx ? 16 : 8, C = V / 8;
  constexpr bool kTurn = V == 16;
  extern __shared__ __align__(16) char slots[];     // quantised: a slot for each group in work
  __shared__ float2 part[6][16];
  __shared__ uint32_t top[16];
  const int lane = threadIdx.x & 63, wave_id = threadIdx.x >> 6;
  const int wave = WAVES == 1 ? 0 : wave_id;
  // 4-bit scales of neighbouring rows share a line: each XCD (workgroup number mod 8) takes rows side by side, so
  // that its L2 puts the line together
  uint32_t block = blockIdx.x;
  if (OUT == kOutMx && (gridDim.x & 7) == 0) block = (block & 7) * (gridDim.x >> 3) + (block >> 3);
  const uint32_t row32 = WAVES == 1 ? block * (blockDim.x >> 6) + wave_id : block;
  if (row32 >= a.M) return;
  const uint32_t mrow32 =
      a.index ? (uint32_t)a.index[row32] : (uint32_t)((uint64_t)row32 * a.each_mul >> a.each_shift);
  if (mrow32 >= a.mod_rows) return;       // of no sequence (negative ones too): the whole row's wavefronts leave
  const int64_t row = row32, mrow = mrow32;
  const int D = a.D;
  auto first = [&](int k) { return ((wave + WAVES * k) * 64 + lane) * V; };

  v8u xr[S][C];
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int c = 0; c < C; ++c) xr[k][c] = load8<kTurn>(a.x + row * a.x_stride, first(k) + 8 * c, D);
  auto rescale = [&](v8u (&raw)[S][C], float by) {
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = widen<kBF16>(raw[k][c][i]) * by;
        raw[k][c] = narrow<kBF16>(p);
      }
  };
  // In fp32 throughout: the residual form's rows, and the quantised ones (fewer instructions than widening
  // where they are read); the plain form into 16 bits waits for memory and keeps its registers.
  constexpr bool kHeld = RES || kTurn;
  float h[kHeld ? S : 1][C][8];
  if constexpr (kHeld && !RES) {
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][c][i] = widen<kBF16>(xr[k][c][i]);
  }
  if constexpr (RES) {
    v8u yr[S][C];
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) yr[k][c] = load8<kTurn>(a.y + row * a.y_stride, first(k) + 8 * c, D);
    float mu = 0.0f, r = 1.0f;
    if (a.post.kind != kNormNone)
      statistics<V, S, WAVES, kBF16>([&](int k, int c, int i) { return widen<kBF16>(yr[k][c][i]); }, first,
                              [&](float by) { rescale(yr, by); }, a.post.kind, a.post.eps, D, a.inv_d, &part[0], mu, r);
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e0 = first(k) + 8 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][c][i] = 0.0f;
        if (e0 >= D) continue;
        float t[8], p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = widen<kBF16>(yr[k][c][i]);
        if (a.post.kind != kNormNone) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = (t[i] - mu) * r;
          if (a.post.weight) {
            load8<kTurn>(a.post.weight, e0, D, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] *= p[i];
          }
          if (a.post.bias) {
            load8<kTurn>(a.post.bias, e0, D, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] += p[i];
          }
        }
        if (a.gate) {
          load_mod<kBF16, kTurn>(a.gate, mrow * a.gate_stride, a.mod_f32, e0, D, p);
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] *= p[i];
        }
        const int left = D - e0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = __fmaf_rn(a.residual_scale, widen<kBF16>(xr[k][c][i]), t[i]);
          h[k][c][i] = kTurn || i < left ? v : 0.0f;
        }
        store8<kTurn>(a.h + row * D, e0, D, narrow<kBF16>(h[k][c]));
      }
  }
  if constexpr (OUT == kOutNone) return;
  auto at = [&](int k, int c, int i) {
    if constexpr (kHeld) return h[k][c][i];
    else return widen<kBF16>(xr[k][c][i]);
  };

  float mu, r;
  statistics<V, S, WAVES, kBF16 || RES>(
      at, first,
      [&](float by) {
        if constexpr (kHeld) {
#pragma unroll
          for (int k = 0; k < S; ++k)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) h[k][c][i] *= by;
        } else {
          rescale(xr, by);
        }
      },
      a.norm.kind, a.norm.eps, D, a.inv_d, &part[3], mu, r);
  float f[kTurn ? (OUT == kOutInt8 ? S : 1) : 1][16];
  const int seg = (int)threadIdx.x >> 4, sl = lane & 15;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    float(&n)[16] = f[OUT == kOutInt8 ? k : 0];
    if constexpr (OUT == kOutInt8) {
#pragma unroll
      for (int i = 0; i < 16; ++i) n[i] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e0 = first(k) + 8 * c;
      if (e0 >= D) continue;
      float t[8], p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = (at(k, c, i) - mu) * r;
      if (a.norm.weight) {
        load8<kTurn>(a.norm.weight, e0, D, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] *= p[i];
      }
      if (a.norm.bias) {
        load8<kTurn>(a.norm.bias, e0, D, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] += p[i];
      }
      if (a.scale) {
        load_mod<kBF16, kTurn>(a.scale, mrow * a.scale_stride, a.mod_f32, e0, D, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __fmaf_rn(t[i], p[i], t[i]);
      }
      if (a.shift) {
        load_mod<kBF16, kTurn>(a.shift, mrow * a.shift_stride, a.mod_f32, e0, D, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] += p[i];
      }
      if constexpr (kTurn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[8 * c + i] = t[i];
      } else {
        store8<kTurn>(static_cast<uint16_t*>(a.values) + row * D, e0, D, narrow<kBF16>(t));
      }
    }
    if constexpr (kTurn) {
      // D is a multiple of 256, so the 16 lanes of a group are all inside or all outside
      if (first(k) < D) {
        rotate_rows(n, slots + seg * kTurnSlot, sl);
        if constexpr (OUT == kOutMx)
          mx_store<4>(n, row, a.M, D, first(k) / kGroup, sl, static_cast<uint8_t*>(a.values),
                      static_cast<uint8_t*>(a.scales));
      }
    }
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
    if (WAVES > 1) {
      if (lane == 0) top[wave] = m;
      __syncthreads();
      m = top[0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) m = max(m, top[w]);
    }
    const bool finite = m < 0x7F800000u;
    const float s = finite ? __uint_as_float(m) / 127.0f : __uint_as_float(0x7FC00000u);
    if (wave == 0 && lane == 0) static_cast<float*>(a.scales)[row] = s * 0.0625f;   // the values are 16 u
#pragma unroll
    for (int k = 0; k < S; ++k)
      if (first(k) < D)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.values) + row * D + first(k)) =
            finite ? codes16(f[k], s) : make_uint4(0, 0, 0, 0);
  }
}

template <bool kBF16, int OUT, bool RES, int S, int WAVES>
hipError_t launch(const NormArgs& a, hipStream_t stream) {
  constexpr bool kTurn = OUT == kOutInt8 || OUT == kOutMx;
  const int rows = WAVES == 1 ? 4 : 1, threads = 64 * WAVES * rows;
  const size_t lds = kTurn ? (size_t)threads / 16 * kTurnSlot : 0;
  const auto fn = &norm_kernel<kBF16, OUT, RES, S, WAVES>;
  if (const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(fn), lds); e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((a.M + rows - 1) / rows), dim3(threads), lds, stream, a);
  return hipGetLastError();
}

// Wavefronts a row and units a lane (a unit is 8 or, quantised, 16 elements).
// Quantised rows have one unit a lane: two are 1 us faster of 32 for 16384 rows
// of 2048 and slower everywhere else (1024 rows 7.7 against 6.1 us, the residual
// form of 16384 rows 70.6 against 65.7).  16-bit outputs have two where that still
// leaves 16 wavefronts a CU (16384 rows of 2048: norm 26.8 against 30.3 us,
// residual 55 against 58), else one, which is faster by latency (1024 rows of 1024:
// norm 4.4 against 4.9 us, residual 5.6 against 6.6).  Four units a lane (residual,
// one wavefront a row of 2048) leave 3 wavefronts a SIMD: 74 us.
template <bool kBF16, int OUT, bool RES>
hipError_t choose(const NormArgs& a, hipStream_t stream) {
  constexpr int V = OUT == kOutInt8 || OUT == kOutMx ? 16 : 8;
  const int units = (a.D + 64 * V - 1) / (64 * V);   // of a wavefront's lanes, over the row
  if (units <= 1) return launch<kBF16, OUT, RES, 1, 1>(a, stream);
  if constexpr (V == 8) {
    if ((int64_t)a.M * units > 4096) {
      if (units <= 2) return launch<kBF16, OUT, RES, 2, 1>(a, stream);
      if (units <= 4) return launch<kBF16, OUT, RES, 2, 2>(a, stream);
      if (units <= 8) return launch<kBF16, OUT, RES, 2, 4>(a, stream);
    }
  }
  if (units <= 2) return launch<kBF16, OUT, RES, 1, 2>(a, stream);
  if (units <= 4) return launch<kBF16, OUT, RES, 1, 4>(a, stream);
  if (units <= 8) return launch<kBF16, OUT, RES, 1, 8>(a, stream);
  if constexpr (V == 8) {
    if (units > 16) return launch<kBF16, OUT, RES, 2, 16>(a, stream);
  }
  return launch<kBF16, OUT, RES, 1, 16>(a, stream);
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
