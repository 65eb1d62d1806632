// Device pieces and plans shared by the attention kernels over the key/value
// cache (internal to the library).
#pragma once

#include "convrot_kv.h"
#include "kv.hpp"

namespace convrot {

// How a call is split: the rows (query, head in group) of one key head in
// tiles of `rows`, the tokens of a sequence in chunks.  A unit is one chunk of
// one sequence.  With balance = 0 every sequence has `splits` units of `chunk`
// tokens (those past its end are idle).  Otherwise the chunk follows from the
// lengths on the device (kv_units), so that the units of all sequences are
// about `balance` per head and tile, and unit numbers run through the
// sequences; `units` bounds them.  Where a sequence may have several units the
// partial outputs go through the workspace: row() numbers them.
struct KvSplit {
  int rows, tiles, kept;     // kept: rows of a tile that can be valid
  int splits, chunk;
  int balance, units;
  KvDivider by_balance;
  float* o;                  // [.., D], unnormalised, rotated basis
  float* ml;                 // [.., 2]: maximum (log2 units) and sum
  __device__ __forceinline__ int64_t row(int h, int tile, int unit, int r) const {
    return (((int64_t)h * tiles + tile) * units + unit) * kept + r;
  }
};
struct KvPlan {
  KvSplit split;
  int64_t parts;             // partial rows
  size_t bytes;              // workspace
  int waves;                 // of a workgroup (few rows)
};

// Workgroups of `waves` wavefronts of the single-token kernel that a CU holds,
// as its registers and LDS are sized, and the wavefronts of a workgroup that
// walks a short context alone.
__host__ __device__ constexpr int kv_decode_wgs(int D, int QT, int waves) {
  return waves > 4 ? 1 : D < 256 ? (QT == 1 ? 4 : 2) : QT == 1 ? 2 : 1;
}
__host__ __device__ constexpr int kv_decode_wide(int D) { return D < 256 ? 16 : 8; }

KvPlan kv_decode_plan(const KvAttn& a);
hipError_t launch_kv_decode(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream);
KvPlan kv_prompt_plan(const KvAttn& a);
hipError_t launch_kv_prompt(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream);
// The finished rows from the splits' partial ones.
hipError_t launch_kv_join(const KvAttn& a, const KvSplit& sp, hipStream_t stream);

// Maximum, and sum, with the lane whose number differs in bit 4 (and in bit 5):
// the two results of a lane swap of v with itself are the pair's two values.
__device__ __forceinline__ float pair32(float v, float& other) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float pair16(float v, float& other) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float max32(float v) {
  float w;
  v = pair32(v, w);
  return fmaxf(v, w);
}
__device__ __forceinline__ float max16_32(float v) {
  float w;
  v = pair16(v, w);
  return max32(fmaxf(v, w));
}
__device__ __forceinline__ float sum32(float v) {
  float w;
  v = pair32(v, w);
  return v + w;
}
__device__ __forceinline__ float sum16_32(float v) {
  float w;
  v = pair16(v, w);
  return sum32(v + w);
}

constexpr float kWeightBits = 8.0f;           // the largest weight is 2^8
constexpr float kUnset = 1e30f;               // base of a row that has seen no token
constexpr float kLowest = -1e30f;             // its maximum
// Before a row's maximum is raised to `best` log2 units.  Weights are 2^(score + base), and fp32 holds scores past
// 2^25 in steps of 4 and more, where their sums with base are no small numbers any more; such a row's factor, and with
// it all of its scores, shrink by a power of two that brings `best` below 2^24.  Its softmax is then flatter by what
// no query's rounding tells apart: weights change where scores differ by less than 2^-16 of the largest.  `best` then
// counts the scores of such a row with log2 scale' = `value` for all of its tokens.  True where a row of the wavefront
// shrank.
__device__ __forceinline__ bool kv_shrink(float& best, float& base, float& factor, float value) {
  const uint32_t e = __float_as_uint(best) >> 23 & 255u;
  const bool far = (e > 127u + 24u) & (kWeightBits - best < base);
  const float by = far ? __uint_as_float((277u - e) << 23) : 1.0f;    // 2^(150 - e)
  factor *= by;
  best = far ? best * by + value : best;
  base = far & (base != kUnset) ? kWeightBits - (kWeightBits - base) * by : base;
  return __any(far);
}
// Raises it, and gives what the row's sums are multiplied by.
__device__ __forceinline__ float kv_raise(float best, float& base) {
  const float was = base;
  base = fminf(was, kWeightBits - best);
  return __builtin_amdgcn_exp2f(base - was);
}
// The row's maximum for the joins, in the units of the factor that it began with.
__device__ __forceinline__ float kv_maximum(float base, float factor, float began) {
  return base == kUnset ? kLowest : factor == began ? kWeightBits - base : (kWeightBits - base) * (began / factor);
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, true);    // row_shr 1, 2, 4, 8
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, true);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, true);    // the row before, into rows 1 and 3
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, true);    // the first half, into the second
  return x;
}

// The units of a balanced call (at most 256 sequences), the same in every
// wavefront of every workgroup: a chunk of `chunk` tokens, a multiple of 128,
// and sequence `b` has units first .. first + n - 1 (n at least 1).  Asked for
// the sequence of a unit (b < 0) or for a sequence; b < 0 on return: no such
// unit.  The chunk starts at the mean that gives `balance` units and, where
// there are at least twice as many units as sequences, grows until the units
// are no more than that, so that they all run at once.  A lane looks at WORDS
// sequences, so all 64 lanes of the wavefront have to call it together.
struct KvUnits {
  int b, first, n, chunk;
  KvSeq seq;
};

template <int WORDS>
__device__ __forceinline__ KvUnits kv_units_of(const KvAttn& a, const KvSplit& sp, int b, int unit) {
  const int lane = threadIdx.x % 64;
  uint32_t blocks[WORDS], n[WORDS], sum[WORDS], mine = 0;
  int kv[WORDS], from[WORDS], to[WORDS];
#pragma unroll
  for (int k = 0; k < WORDS; ++k) {
    const int i = 64 * k + lane;
    const bool in = i < a.batch;
    kv[k] = in ? a.kv_lens[i] : 0;
    from[k] = a.q_start && in ? a.q_start[i] : 0;
    to[k] = a.q_start && in ? a.q_start[i + 1] : 0;
  }
#pragma unroll
  for (int k = 0; k < WORDS; ++k) {
    kv[k] = kv[k] < 0 ? 0 : kv[k] > a.max_kv ? a.max_kv : kv[k];
    blocks[k] = ((uint32_t)kv[k] + 127) / 128;
    mine += blocks[k];
  }
  const uint32_t total = __builtin_amdgcn_readlane(wave_scan(mine), 63), want = (uint32_t)sp.balance;
  uint32_t chunk = kv_divide(total + want - 1, sp.by_balance);   // (2^31 blocks of 128 tokens do not fit the card)
  chunk = chunk < 2 ? 2 : chunk;
  for (;;) {
    // ceil(blocks / chunk) in fp32 (blocks < 2^23): the quotient by the reciprocal is off by one at most
    const float inverse = __builtin_amdgcn_rcpf((float)chunk);
    uint32_t before = 0;
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
      uint32_t need = (uint32_t)((float)blocks[k] * inverse);
      need = need * chunk > blocks[k] ? need - 1 : need;
      need = need * chunk < blocks[k] ? need + 1 : need;
      need = need * chunk < blocks[k] ? need + 1 : need;
      n[k] = 64 * k + lane < a.batch ? (need < 1 ? 1 : need) : 0;
      sum[k] = before + wave_scan(n[k]);
      before = __builtin_amdgcn_readlane(sum[k], 63);
    }
    if (before <= want || 2 * (uint32_t)a.batch > want) break;
    chunk += chunk < 8 ? 1 : chunk / 8;
  }
  KvUnits u{-1, 0, 0, (int)chunk * 128, {0, 0, 0}};
#pragma unroll
  for (int k = WORDS - 1; k >= 0; --k) {
    int at = -1;
    if (b < 0) {
      const uint64_t past = __ballot((64 * k + lane < a.batch) & (sum[k] > (uint32_t)unit));
      if (past) at = __builtin_ctzll(past);
    } else if (b / 64 == k) {
      at = b % 64;
    }
    if (at >= 0) {
      u.b = 64 * k + at;
      u.n = __builtin_amdgcn_readlane(n[k], at);
      u.first = __builtin_amdgcn_readlane(sum[k], at) - u.n;
      int64_t f = (int64_t)u.b * a.each_q, t = f + a.each_q;
      if (a.q_start) {
        f = (int)__builtin_amdgcn_readlane(from[k], at);
        t = (int)__builtin_amdgcn_readlane(to[k], at);
      }
      u.seq = kv_safe(a, f, t, __builtin_amdgcn_readlane(kv[k], at));
    }
  }
  return u;
}
__device__ __forceinline__ KvUnits kv_units(const KvAttn& a, const KvSplit& sp, int b, int unit) {
  return a.batch <= 64 ? kv_units_of<1>(a, sp, b, unit) : kv_units_of<4>(a, sp, b, unit);
}

// The value of the lane whose number in its 16-lane row differs in bit BIT.
template <int BIT>
__device__ __forceinline__ float row_swap(float v) {
  if constexpr (BIT == 0) return dpp_f32<0xB1>(v);                  // quad [1,0,3,2]
  else if constexpr (BIT == 1) return dpp_f32<0x4E>(v);             // quad [2,3,0,1]
  else if constexpr (BIT == 2) return dpp_f32<0x1B>(dpp_f32<0x141>(v));   // i ^ 7, then i ^ 3
  else return dpp_f32<0x128>(v);                                    // rotate the row by 8
}

// x W over 16 lanes with E = D / 16 contiguous elements each (fp32).
template <int D>
__device__ __forceinline__ void rotate_row(float (&x)[D / 16], int seg) {
  constexpr int E = D / 16;
#pragma unroll
  for (int k = 1; k < E; k <<= 1)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if ((i & k) == 0) {
        const float a = x[i], b = x[i + k];
        x[i] = a + b;
        x[i + k] = a - b;
      }
#pragma unroll
  for (int bit = 0; bit < 4; ++bit) {
    const float sign = (seg >> bit) & 1 ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float y = bit == 0 ? row_swap<0>(x[i]) : bit == 1 ? row_swap<1>(x[i]) : bit == 2 ? row_swap<2>(x[i]) : row_swap<3>(x[i]);
      x[i] = __fmaf_rn(x[i], sign, y);
    }
  }
}

// E 16-bit values at p (E = 4, 8 or 16; aligned to 2 E bytes, 16 at most).
template <int E>
__device__ __forceinline__ void load_row(const uint16_t* p, bool bf16, float (&x)[E]) {
  uint32_t w[E / 2];
  if constexpr (E == 4) {
    const v2u r = *reinterpret_cast<const v2u*>(p);
    w[0] = r[0], w[1] = r[1];
  } else {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      const v4u r = reinterpret_cast<const v4u*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = r[j];
    }
  }
  if (bf16) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = in16_f32<false>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
  }
}

template <int E>
__device__ __forceinline__ void store_row(uint16_t* p, bool bf16, const float (&x)[E]) {
  uint32_t w[E / 2];
  if (bf16) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16x2_rn(x[2 * i], x[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pack_f16x2_rn(x[2 * i], x[2 * i + 1]);
  }
  if constexpr (E == 4) {
    *reinterpret_cast<v2u*>(p) = (v2u){w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < E / 8; ++i)
      reinterpret_cast<v4u*>(p)[i] = (v4u){w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
  }
}

}  // namespace convrot
