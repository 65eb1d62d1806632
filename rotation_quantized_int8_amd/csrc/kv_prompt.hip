// Attention of many query rows over the rotated, quantised key/value cache:
// prompts, chunks of prompts, cross attention.
//
// The mathematics is that of the single-token kernel (kv_decode.hip): rotate
// the queries once, use the codes as they are with their scales outside the
// products, rotate the result back.  Here the arithmetic counts, so a
// workgroup of 4 (8) wavefronts takes 128 (256, or 128 with half of the tokens
// each) rows (queries times heads of one group) and shares the decoding: of
// each 64 (128) tokens every wavefront turns the codes of 16 into fp16 (exact)
// and writes them to LDS in the order in which the matrix instructions take
// their operands (16 bytes a lane, no bank conflicts), two buffers deep, so
// that a step costs one barrier.
//   S^T = C_k Q^T     mfma f32 32x32x16 f16, 32 tokens x 32 rows
//   O^T = C_v^T W^T   the same, 32 elements x 32 rows
// A lane owns one row (column lane % 32); the result layout of S^T is the
// operand layout of W^T up to an order of the tokens that C_v^T is stored in.
// The rotated queries are rounded to fp16 after a power of two of the row's
// own, which brings its largest element to 2^9 .. 2^10, far from both ends of
// fp16 (one common to the workgroup spares the product with it below, 2 % of
// the large prompts, but loses a row next to one 2^16 times as loud).  For
// fp16 rows the remainder, rounded again, takes a second product into the same
// accumulator: left out, it would cost the outputs twice their own rounding
// (measured: 4.1e-4 against 2.1e-4, with it 2.8e-4); next to the rounding of a
// bf16 output it is nothing.  The weights are rounded to fp16 (2^-11 of each
// at most, to nearest), so a sum of many is off by less than the output's own
// rounding.  sm_scale and log2 e are multiplied into the keys' scales, so a
// weight is exp2(fma(S, scale_j unit_row, base_row)): two operations, its
// exponential, its share of the sum and the product with the value's scale.
// The running maximum is raised only when a weight could pass 2^15 (they start
// at 2^8 for the largest).
//
// What bounds it: the vector work on the weights (six operations a weight,
// the exponential at a quarter of the rate) next to the matrix products, which
// the two wavefronts of a SIMD overlap only in part.  Measured: 4096 causal
// queries of 32 heads over 8 key heads, D 128, bf16, 4 bits: 174 us, 790
// TFLOP/s, against 1220 of a large matrix product; three chunks of up to 701
// queries, 24 heads over 8, D 64, fp16, 8 bits, contexts of up to 6007: 134
// us, 330 TFLOP/s (the remainder's product is not counted); 1024 queries of 16
// heads over 512 states, twice: 26.5 us.  Three wavefronts a SIMD for heads of
// 128, steps of 32 tokens, the two halves of a step offset between the
// wavefronts, and the next scores formed before the outputs were no faster.
// Heads of 256 hold 128 (fp16: 192) registers of outputs and queries before
// anything else and run one wavefront a SIMD, with what does not fit in the
// accumulation registers: 2048 x 2048 causal, 16 heads over 8, fp16, 4 bits,
// 147 us, 234 TFLOP/s; 256 rows over 4 x 8192, 8 heads, 186 us.

#include "kv_core.hpp"
#include "launch.hpp"

namespace convrot {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr float kMostWeight = 32768.0f;
constexpr float kLeastScale = 0x1p-80f;       // as in the single-token kernel
constexpr float kMostSum = 0x1p92f;

// a b, and 0 where a is 0 whatever b is.
__device__ __forceinline__ float mul_legacy(float a, float b) {
  float d;
  asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}

__device__ __forceinline__ uint32_t less(uint32_t x, float by) {
  const h2 off = {(_Float16)by, (_Float16)by};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, x) - off);
}

// The eight elements of unit (8 codes) a next to those of unit b, as half
// pairs (4 bits: the odd elements times 16): 1024 + (c + 8) and the like by a
// mask and an exclusive or, less 1032.  Two units of one token make a key
// operand, one unit of two tokens a value operand.
template <int BITS>
__device__ __forceinline__ void halves(const uint32_t* a, const uint32_t* b, uint32_t (&f)[8]) {
  if constexpr (BITS == 4) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const uint32_t x = __builtin_amdgcn_perm(b[0], a[0], i ? 0x07060302u : 0x05040100u), y = x >> 8;
      f[i] = less((x & 0x000F000Fu) ^ 0x64086408u, 1032.0f);
      f[i + 1] = less((x & 0x00F000F0u) ^ 0x64806480u, 1152.0f);
      f[i + 2] = less((y & 0x000F000Fu) ^ 0x64086408u, 1032.0f);
      f[i + 3] = less((y & 0x00F000F0u) ^ 0x64806480u, 1152.0f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = less(__builtin_amdgcn_perm(b[i / 4], a[i / 4], 0x0C040C00u + (uint32_t)(i % 4) * 0x00010001u) ^ 0x64806480u,
                  1152.0f);
  }
}

// HALVES = 2: two wavefronts share 32 rows, each takes half of a step's tokens.
template <int D, int BITS, int WAVES, int HALVES>
struct Prompt {
  static constexpr int kGroups = WAVES / HALVES;       // of 32 rows
  static constexpr int kThreads = 64 * WAVES, kRows = 32 * kGroups;
  static constexpr int kStep = 16 * WAVES;             // tokens of a step: each wavefront decodes a group of 16
  static constexpr int kRow = D * BITS / 8;            // bytes of a cached row
  static constexpr int kUnit = BITS;                   // bytes of 8 codes
  static constexpr int kUnits = D / 8;
  static constexpr int kSteps = D / 16;                // matrix steps of a score
  static constexpr int kTiles = D / 32;                // output tiles
  static constexpr int kSpread = 256 / D;              // elements of a unit that share an output tile
  // A wavefront's group of 16 tokens: 16-byte pieces of the keys' rows, and units of 4 tokens of the values'.
  static constexpr int kPieces = kRow, kTasks = 4 * kUnits;
  static constexpr int kKeyEach = kPieces < 64 ? 1 : kPieces / 64;
  static constexpr int kValueEach = kTasks < 64 ? 1 : kTasks / 64;
  static constexpr int kBuffer = kStep * D * 2;        // bytes of a step's keys, and of its values
  static constexpr int kBytes = 4 * kBuffer;
};

template <int D, int BITS, int WAVES, int HALVES, bool BF16>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : D == 64 && HALVES == 1 ? 3 : 2)
void kv_prompt_kernel(KvAttn a, KvSplit sp) {
  using P = Prompt<D, BITS, WAVES, HALVES>;
  constexpr int kRows = P::kRows, kStep = P::kStep;
  extern __shared__ __align__(16) char lds[];          // keys [2], values [2]
  __shared__ __align__(16) float kscale[2][kStep], vscale[2][kStep];
  __shared__ __align__(16) int absent[2][WAVES];
  __shared__ __align__(16) float vtop[2][WAVES];      // largest value scale of each group
  __shared__ float began[WAVES][32];                   // the rows' units

  const int tid = threadIdx.x, lane = tid % 64, col = lane % 32, hi = lane / 32;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int group = HALVES == 1 ? wave : wave % P::kGroups, half = HALVES == 1 ? 0 : wave / P::kGroups;   // of rows, and of a step's tokens
  const int b = blockIdx.z;
  // the key head is the fastest index, so that the workgroups of one head meet in one XCD's L2 where the head
  // count is a multiple of 8; the last tiles, which see the most tokens, start first
  const int h = blockIdx.x % a.c.heads;
  const int rest = blockIdx.x / a.c.heads;
  const int split = rest % sp.splits, tile = sp.tiles - 1 - rest / sp.splits;
  const int log2p = a.c.page_log2;
  const int c0 = split * sp.chunk;

  const KvSeq s = kv_sequence(a, b);
  const int rows = s.n * a.group - tile * kRows;
  if (rows <= 0) return;
  const int last = a.causal ? s.kv - s.n + kv_query_of(a, tile * kRows + (rows < kRows ? rows : kRows) - 1) + 1 : s.kv;
  const int c1 = last < c0 + sp.chunk ? last : c0 + sp.chunk;
  if (c1 <= c0 && split > 0) return;

  // ---- raw codes and scales of the wavefront's next group, in registers.  Its page numbers of 64 steps are held a
  // lane each; the group's first row is uniform.
  v4u rawk[P::kKeyEach];
  uint32_t rawv[P::kValueEach][4][P::kUnit / 4];
  float raws;
  int pages, present = 0;
  auto find_pages = [&](int step) {
    const int64_t j = c0 + (int64_t)kStep * (step + lane) + 16 * wave;
    const int p = j < c1 ? a.table[b * a.width + (j >> log2p)] : -1;
    pages = p < a.c.pages ? p : -1;
  };
  const uint32_t koff = lane % 16 * P::kRow + lane / 16 % (P::kRow / 16) * 16;
  auto load = [&](int step) __attribute__((always_inline)) {
    if (step % 64 == 0) find_pages(step);
    const int j = c0 + kStep * step + 16 * wave, p = __builtin_amdgcn_readlane(pages, step % 64);
    present = p >= 0;
    const int64_t row = (((int64_t)(p < 0 ? 0 : p) * a.c.heads + h) << log2p) + (j & ((1 << log2p) - 1));
    uint32_t key = koff;                               // (opaque: the compiler would keep kc + koff, two registers a lane)
    asm volatile("" : "+v"(key));
    const uint8_t* kbase = a.c.kc + row * P::kRow;
    const uint8_t* vbase = a.c.vc + row * P::kRow;
#pragma unroll
    for (int i = 0; i < P::kKeyEach; ++i) rawk[i] = *reinterpret_cast<const v4u*>(kbase + (key + i * 64));
#pragma unroll
    for (int i = 0; i < P::kValueEach; ++i) {
      const int task = (lane + 64 * i) % P::kTasks;
      const uint32_t off = task / P::kUnits * 4 * P::kRow + task % P::kUnits * P::kUnit;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int w = 0; w < P::kUnit / 4; ++w)
          rawv[i][t][w] = reinterpret_cast<const uint32_t*>(vbase + (off + t * P::kRow))[w];
    }
    raws = (lane < 16 ? a.c.ks : a.c.vs)[row + lane % 16];
  };
  if (c1 > c0) load(0);

  // ---- the rotated queries as fp16.  The rotation is a matrix product too: W (+-1, exact) times the rows, whose
  // result layout is, in pairs of registers, the operand layout of the scores: lane (column = row, hi), step k, holds
  // elements 4 hi .. 4 hi + 3 of units 2 k and 2 k + 1, alternating.
  const int myrow = tile * kRows + 32 * group + col, myquery = kv_query_of(a, myrow);
  // what a score's product is multiplied by: sm_scale, the rotation's 1 / sqrt(D) and log2 e, in the keys' scales (the
  // sign of sm_scale is the queries'), and the unit of this lane's row
  const float common = fabsf(a.scale) * kv_rsqrt(D) * 1.44269504088896340736f;
  float unit;
  v8h q[P::kSteps], left_over[BF16 ? 1 : P::kSteps];        // fp16 rows: and what the rounding leaves
  {
    v16f x[P::kTiles];
#pragma unroll
    for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) x[t][r] = 0.0f;
    // W's operand of tile t, step k: the sign of element (m, d), m = 32 t + col, d = 16 k + 8 hi + j, is the parity of
    // m & d = that of (col & 7) & j, of (col >> 3 & hi & 1), of (col >> 4) & k & 1 and of t & (k >> 1)
    const uint32_t one = BF16 ? 0x3F80u : 0x3C00u;
    v4u w[2][2];                                       // by k & 1, and negated
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (uint32_t)__builtin_popcount(col & 7 & 2 * i), up = (uint32_t)__builtin_popcount(col & 7 & (2 * i + 1));
      const uint32_t pair = one * 0x00010001u ^ (lo & 1) << 15 ^ (up & 1) << 31;
      w[0][0][i] = pair ^ (col >> 3 & hi & 1 ? 0x80008000u : 0u);
      w[1][0][i] = w[0][0][i] ^ (col >> 4 ? 0x80008000u : 0u);
      w[0][1][i] = w[0][0][i] ^ 0x80008000u;
      w[1][1][i] = w[1][0][i] ^ 0x80008000u;
    }
    const bool in = myquery < s.n;
    const uint16_t* src = a.q.p + (in ? (s.first + myquery) * a.q.token + (h * a.group + myrow - myquery * a.group) * a.q.head : 0);
    v4u raw[P::kSteps];
#pragma unroll
    for (int k = 0; k < P::kSteps; ++k) {
      raw[k] = *reinterpret_cast<const v4u*>(src + 8 * (2 * k + hi));
      if (!in) raw[k] = (v4u){0, 0, 0, 0};
    }
#pragma unroll
    for (int k = 0; k < P::kSteps; ++k)
#pragma unroll
      for (int t = 0; t < P::kTiles; ++t) {
        const v4u sign = w[k & 1][__builtin_popcount(t & k >> 1) & 1];
        if constexpr (BF16)
          x[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, sign), __builtin_bit_cast(v8b, raw[k]), x[t], 0, 0, 0);
        else
          x[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, sign), __builtin_bit_cast(v8h, raw[k]), x[t], 0, 0, 0);
      }
    float top = 0.0f;
#pragma unroll
    for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[t][r]));
    top = max32(top);
    // (a row with an infinity or a NaN has no finite element, and shows NaN)
    const uint32_t e2 = __float_as_uint(top) >> 23;
    unit = top < INFINITY ? __uint_as_float((e2 < 10u ? 1u : e2 - 9u) << 23) : __uint_as_float(0x7FC00000u);
    if (hi == 0) began[wave][col] = unit;              // (read by the same wavefront)
    const float by = (a.scale < 0.0f ? -1.0f : 1.0f) / unit, odd = BITS == 4 ? by * 0.0625f : by;
#pragma unroll
    for (int k = 0; k < P::kSteps; ++k) {
      v4u y, z;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * (k % 2) + i;
        const float f = x[k / 2][r] * (i % 2 ? odd : by), g = x[k / 2][r + 4] * (i % 2 ? odd : by);
        y[i] = pack_f16x2_rn(f, g);
        const h2 near = __builtin_bit_cast(h2, (uint32_t)y[i]);
        z[i] = pack_f16x2_rn(f - (float)near[0], g - (float)near[1]);
      }
      q[k] = __builtin_bit_cast(v8h, y);
      if constexpr (!BF16) left_over[k] = __builtin_bit_cast(v8h, z);
    }
  }

  char* kbuf = lds;
  char* vbuf = lds + 2 * P::kBuffer;
  auto decode = [&](int buf, int step) __attribute__((always_inline)) {
    if (P::kPieces >= 64 || lane < P::kPieces) {
      char* dst = kbuf + buf * P::kBuffer + ((wave / 2) * P::kSteps * 64 + wave % 2 * 16 + lane % 16) * 16;
#pragma unroll
      for (int i = 0; i < P::kKeyEach; ++i)
#pragma unroll
        for (int n = 0; n < 16 / P::kUnit; n += 2) {
          uint32_t w[16 / 4], f[8];
#pragma unroll
          for (int z = 0; z < 4; ++z) w[z] = rawk[i][z];
          halves<BITS>(w + n * (P::kUnit / 4), w + (n + 1) * (P::kUnit / 4), f);
          const int step2 = ((4 * i + lane / 16 % (P::kRow / 16)) * (16 / P::kUnit) + n) / 2;
          *reinterpret_cast<v4u*>(dst + step2 * 1024) = (v4u){f[0], f[1], f[2], f[3]};
          *reinterpret_cast<v4u*>(dst + step2 * 1024 + 512) = (v4u){f[4], f[5], f[6], f[7]};
        }
    }
    if (P::kTasks >= 64 || lane < P::kTasks) {
#pragma unroll
      for (int i = 0; i < P::kValueEach; ++i) {
        const int task = lane + 64 * i, quad = task / P::kUnits, unit = task % P::kUnits;
        uint32_t f01[8], f23[8];
        halves<BITS>(rawv[i][0], rawv[i][1], f01);
        halves<BITS>(rawv[i][2], rawv[i][3], f23);
        // tokens 16 wave + 8 half + 4 g + 0..3: operand `wave`, lanes of half-wave g, its half `half`
        const int half = quad / 2, g = quad % 2;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = e / P::kSpread, row = e % P::kSpread * P::kUnits + unit;
          *reinterpret_cast<v2u*>(vbuf + buf * P::kBuffer + ((t * WAVES + wave) * 64 + g * 32 + row) * 16 + half * 8) =
              (v2u){f01[e], f23[e]};
        }
      }
    }
    const int j = c0 + kStep * step + 16 * wave + lane % 16;
    const float v = (j < c1) & (present != 0) ? raws : 0.0f, most = warp_max16(v);
    // a value's scale of NaN (lanes 32 on hold the values' too) makes its key's one, so that it shows in every row that
    // sees the token, however small its weight
    float value;
    pair32(raws, value);
    if (lane < 16) {
      kscale[buf][16 * wave + lane] = value == value ? raws * common : value;
    } else if (lane < 32) {
      vscale[buf][16 * wave + lane - 16] = v;
      if (lane == 16) {
        vtop[buf][wave] = most;
        absent[buf][wave] = !present;
      }
    }
  };

  // ---- the steps
  const int end = myquery >= s.n ? 0 : a.causal ? s.kv - s.n + myquery + 1 : s.kv;
  const int first = a.causal ? s.kv - s.n + kv_query_of(a, tile * kRows + 32 * group) + 1 : s.kv;   // the wavefront's first row
  v16f o[P::kTiles];
  float base = kUnset, l = 0.0f;
#pragma unroll
  for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[t][r] = 0.0f;

  auto score = [&](int buf, int kt) __attribute__((always_inline)) {
    v16f z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.0f;
#pragma unroll
    for (int k = 0; k < P::kSteps; ++k) {
      const v8h c = *reinterpret_cast<const v8h*>(kbuf + buf * P::kBuffer + ((kt * P::kSteps + k) * 64 + lane) * 16);
      z = __builtin_amdgcn_mfma_f32_32x32x16_f16(c, q[k], z, 0, 0, 0);
      if constexpr (!BF16) z = __builtin_amdgcn_mfma_f32_32x32x16_f16(c, left_over[k], z, 0, 0, 0);
    }
    return z;
  };
  // the 32 tokens from j on, whose products with the queries are z: weights, then outputs
  auto use = [&](int buf, int kt, int j, v16f z) __attribute__((always_inline)) {
    const v2u gone = *reinterpret_cast<const v2u*>(&absent[buf][2 * kt]);
    const bool whole = __builtin_amdgcn_readfirstlane((j + 32 <= first) & !(gone[0] | gone[1]));
    const int left = end - j - 4 * hi;                 // (one register, where the compiler would keep sixteen bounds)
    auto seen = [&](int r) { return (8 * (r / 4) + r % 4 < left) & !gone[r / 8]; };
    const float vmost = fmaxf(vtop[buf][2 * kt], vtop[buf][2 * kt + 1]);
    float sum;
    for (bool again = false;; again = true) {          // z becomes the weights
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const v4f ks = *reinterpret_cast<const v4f*>(&kscale[buf][32 * kt + 2 * r + 4 * hi]);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[r + i] = __builtin_amdgcn_exp2f(__fmaf_rn(z[r + i], ks[i] * unit, base));
      }
      if (!whole) {
#pragma unroll
        for (int r = 0; r < 16; ++r) z[r] = seen(r) ? z[r] : 0.0f;
      }
      sum = ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
      sum += ((z[8] + z[9]) + (z[10] + z[11])) + ((z[12] + z[13]) + (z[14] + z[15]));
      // raise the maximum (rare) where a weight might pass 2^15; a row that has seen no token has an infinite sum
      if (again || !__any((sum * vmost > kMostWeight) | (sum > kMostSum))) break;
      z = score(buf, kt);
      float best = kLowest;
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const v4f ks = *reinterpret_cast<const v4f*>(&kscale[buf][32 * kt + 2 * r + 4 * hi]);
        const v4f vs = *reinterpret_cast<const v4f*>(&vscale[buf][32 * kt + 2 * r + 4 * hi]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = z[r + i] * (ks[i] * unit) + __builtin_amdgcn_logf(fmaxf(vs[i], kLeastScale));
          best = fmaxf(best, (whole | seen(r + i)) ? y : kLowest);
        }
      }
      best = max32(best);
      kv_shrink(best, base, unit, __builtin_amdgcn_logf(fmaxf(vmost, kLeastScale)));
      const float by = kv_raise(best, base);
      l *= by;
#pragma unroll
      for (int t = 0; t < P::kTiles; ++t) o[t] *= by;
    }
    // times the values' scales; a weight of 0 stays 0 under a NaN scale, which another row may see
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const v4f vs = *reinterpret_cast<const v4f*>(&vscale[buf][32 * kt + 2 * r + 4 * hi]);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[r + i] = mul_legacy(z[r + i], vs[i]);
    }
    l += sum;
    v4u w[2];
#pragma unroll
    for (int r = 0; r < 16; r += 2) w[r / 8][r % 8 / 2] = pack_f16x2_rn(z[r], z[r + 1]);
#pragma unroll
    for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const v8h c = *reinterpret_cast<const v8h*>(vbuf + buf * P::kBuffer + ((t * WAVES + 2 * kt + u) * 64 + lane) * 16);
        o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(c, __builtin_bit_cast(v8h, w[u]), o[t], 0, 0, 0);
      }
  };

  if (c1 > c0) {
    decode(0, 0);
    if (c0 + kStep < c1) load(1);
    __syncthreads();
    int buf = 0, step = 0;
    for (int j = c0; j < c1; j += kStep, buf ^= 1, ++step) {
      if (j + kStep < c1) {
        decode(buf ^ 1, step + 1);
        if (j + 2 * kStep < c1) load(step + 2);
      }
#pragma unroll
      for (int n = 0; n < P::kGroups / 2; ++n) {
        const int kt = P::kGroups / 2 * half + n;
        if (j + 32 * kt >= c1) break;
        use(buf, kt, j + 32 * kt, score(buf, kt));
      }
      __syncthreads();
    }
  }

  l = sum32(l);
  float most = kv_maximum(base, unit, began[wave][col]);
  if constexpr (HALVES == 2) {                         // the second half's outputs join the first's
    v4f* far = reinterpret_cast<v4f*>(lds) + 64 * group + lane;
    float* rest_of = reinterpret_cast<float*>(lds + P::kTiles * 4 * P::kGroups * 1024) + 2 * (64 * group + lane);
    if (half) {
#pragma unroll
      for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          far[(4 * t + r / 4) * P::kGroups * 64] = (v4f){o[t][r], o[t][r + 1], o[t][r + 2], o[t][r + 3]};
      rest_of[0] = most;
      rest_of[1] = l;
    }
    __syncthreads();
    if (half) return;
    const float other = rest_of[0], top = fmaxf(most, other);
    const float mine = __builtin_amdgcn_exp2f(most - top), its = __builtin_amdgcn_exp2f(other - top);
    l = l * mine + rest_of[1] * its;
#pragma unroll
    for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const v4f y = far[(4 * t + r / 4) * P::kGroups * 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][r + i] = o[t][r + i] * mine + y[i] * its;
      }
    most = top;
  }
  // ---- a lane holds half a row: rotate it back (every bit of (tile, register) and the half-wave is a bit of the
  // element's number), or leave it to the join
  if (myquery >= s.n || 32 * group + col >= rows) return;
  // element of (tile t, register r): row = 8 (r / 4) + 4 hi + r % 4, unit = row % kUnits, e = t * kSpread + row / kUnits
  auto unit_of = [&](int r) { return (8 * (r / 4) + 4 * hi + r % 4) % P::kUnits; };
  auto e_of = [&](int t, int r) { return t * P::kSpread + 8 * (r / 4) / P::kUnits; };
  float x[P::kTiles * 16];
  const float by = sp.splits > 1 ? 1.0f : l == 0.0f ? 0.0f : kv_rsqrt(D) / l;
#pragma unroll
  for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      x[16 * t + r] = l == 0.0f ? 0.0f : o[t][r] * (BITS == 4 && e_of(t, r) % 2 ? by * 0.0625f : by);
  // the lane's units, 8 elements each
  auto units = [&](auto&& store) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < 2 * P::kTiles; ++n) {
      float y[8];
      int unit = 0;
#pragma unroll
      for (int t = 0; t < P::kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (r % 4 + 4 * (r / 4 % (P::kUnits / 8)) == n) {
            y[e_of(t, r)] = x[16 * t + r];
            unit = unit_of(r);
          }
      store(unit, y);
    }
  };
  if (sp.splits > 1) {
    const int64_t at = sp.row(h, tile, b * sp.splits + split, 32 * group + col);
    float* dst = sp.o + at * D;
    units([&](int unit, float (&y)[8]) {
      *reinterpret_cast<v4f*>(dst + 8 * unit) = (v4f){y[0], y[1], y[2], y[3]};
      *reinterpret_cast<v4f*>(dst + 8 * unit + 4) = (v4f){y[4], y[5], y[6], y[7]};
    });
    if (hi == 0) {
      sp.ml[2 * at] = most;
      sp.ml[2 * at + 1] = l;
    }
    return;
  }
#pragma unroll
  for (int k = 1; k < P::kTiles * 16; k <<= 1)
#pragma unroll
    for (int i = 0; i < P::kTiles * 16; ++i)
      if ((i & k) == 0) {
        const float y = x[i], z = x[i + k];
        x[i] = y + z;
        x[i + k] = y - z;
      }
#pragma unroll
  for (int i = 0; i < P::kTiles * 16; ++i) {
    float second;
    const float one = pair32(x[i], second);
    x[i] = hi ? one - second : one + second;
  }
  const int head = h * a.group + myrow - myquery * a.group;
  uint16_t* dst = a.o + ((s.first + myquery) * a.q_heads + head) * D;
  units([&](int unit, float (&y)[8]) { store_row<8>(dst + 8 * unit, BF16, y); });
}

template <int D, int BITS, int WAVES, int HALVES, bool BF16>
hipError_t run(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  KvSplit sp = p.split;
  sp.o = static_cast<float*>(workspace);
  sp.ml = sp.o ? sp.o + p.parts * D : nullptr;
  const auto fn = kv_prompt_kernel<D, BITS, WAVES, HALVES, BF16>;
  const size_t lds = Prompt<D, BITS, WAVES, HALVES>::kBytes;
  if (hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(fn), lds)) return e;
  fn<<<dim3((unsigned)(a.c.heads * sp.splits * sp.tiles), 1, a.batch), 64 * WAVES, lds, stream>>>(a, sp);
  if (hipError_t e = hipGetLastError()) return e;
  return sp.splits > 1 ? launch_kv_join(a, sp, stream) : hipSuccess;
}

template <int BITS, bool BF16>
hipError_t run(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  if (a.c.head_dim == 256) return run<256, BITS, 4, 1, BF16>(a, p, workspace, stream);
  if (a.c.head_dim == 64)
    return p.waves == 8 ? run<64, BITS, 8, 2, BF16>(a, p, workspace, stream) : run<64, BITS, 4, 1, BF16>(a, p, workspace, stream);
  if (p.waves == 8 && p.split.rows == 128) return run<128, BITS, 8, 2, BF16>(a, p, workspace, stream);
  return p.waves == 8 ? run<128, BITS, 8, 1, BF16>(a, p, workspace, stream) : run<128, BITS, 4, 1, BF16>(a, p, workspace, stream);
}

template <int BITS>
hipError_t run(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  return a.bf16 ? run<BITS, true>(a, p, workspace, stream) : run<BITS, false>(a, p, workspace, stream);
}

}  // namespace

// Heads of 128 with enough rows take workgroups of 8 wavefronts for 256 rows,
// which halves the decoding a row (4096 x 4096 causal, 32 heads: 190 us
// against 210 us).  Where tiles of 128 rows leave at most one workgroup for a
// CU, 8 wavefronts share them, two to 32 rows, each half of the tokens, so
// that a SIMD still has two (1024 x 1024 causal, 32 heads over 8: 33.6 us
// against 44.8 with 4 wavefronts; 1024 x 2048, 16 heads, twice: 60 against
// 85).  They join for 2 us, so not for contexts of one step (64 x 64: 12.8
// against 10.5), nor for long contexts of several sequences, where splitting
// evens out their lengths (five of 150 queries over up to 8000 tokens: 174
// against 139).
// The tokens are split where the workgroups leave room for more: one sequence
// into as many units as run at once (3000 x 3000, heads of 64: 96 us, twice
// as many 122 us), several into two rounds, which evens out unequal lengths
// (three sequences of 700 queries over 6000 tokens: one split 190 us, three
// 150 us, five 177 us).
KvPlan kv_prompt_plan(const KvAttn& a) {
  KvPlan p{};
  const int64_t rows = (int64_t)a.max_q * a.group;
  KvSplit& s = p.split;
  const int64_t heads = (int64_t)a.c.heads * a.batch;
  const bool shared = a.c.head_dim < 256 && a.max_kv > 128 && (a.batch == 1 || a.max_kv <= 2048) &&
                      (rows + 127) / 128 * heads <= 256;
  const bool tall = a.c.head_dim == 128 && (rows + 255) / 256 * heads >= 256;
  p.waves = shared || tall ? 8 : 4;
  s.rows = tall ? 256 : 128;
  s.tiles = (int)((rows + s.rows - 1) / s.rows);
  s.kept = (int)(rows < s.rows ? rows : s.rows);
  const int64_t base = s.tiles * heads;
  const int64_t slots = p.waves == 8 || a.c.head_dim == 256 ? 256 : a.c.head_dim == 128 ? 512 : 768;   // resident
  int64_t splits = (a.batch > 1 && !shared ? 2 : 1) * slots / base;
  const int64_t most = ((int64_t)a.max_kv + 511) / 512;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  const int64_t chunk = (a.max_kv + splits - 1) / splits, step = 16 * p.waves;
  s.chunk = (int)((chunk + step - 1) / step * step);
  if (s.chunk < step) s.chunk = (int)step;
  s.splits = (int)(((int64_t)a.max_kv + s.chunk - 1) / s.chunk);
  if (s.splits < 1) s.splits = 1;
  s.units = (int)(a.batch * s.splits);
  p.parts = s.splits > 1 ? base * s.splits * s.kept : 0;
  p.bytes = (size_t)p.parts * (a.c.head_dim + 2) * 4;
  return p;
}

hipError_t launch_kv_prompt(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  return a.c.bits == 4 ? run<4>(a, p, workspace, stream) : run<8>(a, p, workspace, stream);
}

}  // namespace convrot
