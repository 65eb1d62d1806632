// Attention of few query rows over the rotated, quantised key/value cache:
// single tokens, and the join of a sequence's splits.
//
// Mathematics.  H is orthonormal and symmetric, so q . k = (q H) . (k H): the
// query row is rotated once, the cached codes c are used as they are, and only
// the finished output row is rotated back.  With the row's softmax weight p_j,
//   score_j = sm_scale scale_j (q H) . c_j,     o = (sum_j p_j scale'_j c'_j / sum_j p_j) H.
//
// Both products run on the matrix cores with the keys' and values' codes as
// the left operand, so that a lane owns one query row (column lane % 16 of
// the result) throughout:
//   S^T = C_k Q^T   mfma i32 16x16x64 i8.  The rotated query is held as 16-bit
//                   fixed point of its own maximum in two int8 planes,
//                   q = 256 hi + lo, so the product is exact; a 4-bit code
//                   enters as 16 c (its nibble moved to the upper half of a
//                   byte, one AND or a shift and an AND for four codes).
//   O^T = C_v^T W^T mfma f32 16x16x32 f16.  The result layout of S^T (rows
//                   4 (lane / 16) + r) is the operand layout of W^T, so the
//                   weights never leave their lane; a lane loads, for each of
//                   its 8 tokens, the D / 16 codes of its own D / 16 elements
//                   and interleaves pairs of tokens by byte permutes.
// W = p scale' with p = 2^(score - m + 8) and m the running maximum of
// score + log2 scale', so fp16 keeps weights down to 2^-32 of the largest.
// For fp16 outputs what their rounding leaves takes a second product: left
// out, it costs few rows up to the outputs' own rounding again (error 2.0 times
// the plain form's at worst over 700 draws, with it 1.1; one token over 1000
// 12.4 -> 12.8 us, larger calls level).  Next to a bf16 output's it is nothing.
// m is raised only when a weight passes 2^15, so most steps neither reduce
// over lanes nor rescale, and no maximum is needed before the exponential.
// The values' codes enter with an offset of 8 or 128 (see value_operands), so
// the sums round at 2^-24 of 8 (128) sum W where even tokens leave a mean that
// is smaller than sum W by sqrt(tokens).  The offset is taken off every 64 steps
// (2048 tokens), which keeps that at 5e-5 of an output over 131072 tokens in
// one workgroup; taken off at the end alone it comes to 4e-4.
//
// What bounds it: HBM (each cached row is read once for up to 32 rows of its
// key head).  A workgroup of 4 wavefronts owns one chunk of the tokens of one
// sequence and key head; the wavefronts take 32 tokens in turn.  Codes and
// scales come by direct loads into a ring in LDS of the wavefront's own, two
// steps deep or one, so loads in flight cost no registers
// and the loop needs no barrier.
//
// Measured, against the time of a copy of as many bytes at 5.1 TB/s: 32
// sequences of up to 8192 tokens, 8 key heads of 4 query heads, D 128, 4 bits
// (174 MB): 38.7 us and 5.3 us for the join (4.5 TB/s in the kernel); two
// sequences of 131072 tokens, 4 key heads of 8 (143 MB): 30 and 5.2 us (4.7
// TB/s); 48 of up to 2501 tokens, 4 key heads of 5, D 256, 8 bits (164 MB):
// 41 us in one launch (4.0 TB/s).  One token over 1000 of 16 heads: 13 us, the
// latency of the prologue, two steps and the join of 16 wavefronts (split over
// more workgroups and joined by a second launch it is as fast in a graph and
// slower in a stream of single calls, see the plan).
// What is left to the copy's rate is the start (lengths, pages, the rotation
// of the queries, about 4 us a workgroup before the first product) and the
// vector work of a step, which a SIMD's four wavefronts overlap with loads
// only in part.

#include "dma.hpp"
#include "kv_core.hpp"

namespace convrot {
namespace {

constexpr int kStep = 32;                     // tokens a wavefront takes at once
constexpr float kMostWeight = 32768.0f;       // m is raised past this weight
constexpr float kLeastScale = 0x1p-80f;       // a value's scale in the maximum, at least
constexpr float kMostSum = 0x1p92f;           // and past this sum of a step: only values of almost 0 get there

// The ring of a wavefront in LDS: kStages steps of 32 tokens, each the keys'
// codes, the values' codes and the scales (keys' then values', 16 each).  One
// step where two would keep a fourth (a second, for heads of 256) workgroup
// off the CU.
template <int D, int BITS>
struct Ring {
  static constexpr int kRow = D * BITS / 8;            // bytes of a cached row
  static constexpr int kHalf = kStep * kRow;           // of a step's keys, and of its values
  static constexpr int kStage = 2 * kHalf + 4 * 64;
  static constexpr int kStages = kRow > 128 || D * BITS == 1024 && D < 256 ? 1 : 2;
  static constexpr int kBytes = kStages * kStage;
  static constexpr int kLoads = kHalf / 1024;          // direct loads of a half
  static constexpr int kKeyWords = kRow / 16;          // 32-bit words of a lane's key codes (16 tokens, 4 lanes each)
  static constexpr int kValueWords = kRow < 64 ? 1 : kRow / 64;
};

// S^T operand k of 16 tokens, 16 int8 a lane.  w: the lane's codes, the 16
// bytes (lane / 16) of each 64 of its token's row (8 bytes of 32 where a row
// has 32).  A 4-bit code enters as 16 c: the even elements of the 32 that 16
// bytes hold, then the odd ones.
template <int D, int BITS>
__device__ __forceinline__ v4i key_operand(const uint32_t* w, int k) {
  v4i a;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BITS == 8) {
      a[j] = (int)w[4 * k + j];
    } else if constexpr (D == 64) {
      a[j] = (int)(j < 2 ? (w[j] << 4) & 0xF0F0F0F0u : w[j - 2] & 0xF0F0F0F0u);
    } else {
      const uint32_t x = w[4 * (k / 2) + j];
      a[j] = (int)(k % 2 == 0 ? (x << 4) & 0xF0F0F0F0u : x & 0xF0F0F0F0u);
    }
  }
  return a;
}

// Where element d of a query stands among its D int8, so that lane quad reads
// the D / 4 from quad * D / 4 on in the order of the key operands.
template <int D, int BITS>
__device__ __forceinline__ constexpr int query_place(int d) {
  const int byte = d * BITS / 8;                       // of a cached row
  if (BITS == 8) return byte / 16 % 4 * (D / 4) + byte / 64 * 16 + byte % 16;
  if (D == 64) return byte / 8 * 16 + d % 2 * 8 + byte % 8;
  return byte / 16 % 4 * (D / 4) + byte / 64 * 32 + d % 2 * 16 + byte % 16;
}

// O^T operands of output tiles i .. i + 3: of 8 tokens' words, four half pairs
// a tile.  A code enters as the fp16 number whose bits are c + 8 (c + 128 for
// 8 bits), a subnormal, and the sum of the weights times the offset is taken
// off later.  4 bits enter 6 bits up, as (c + 8) 2^-18: the products of a
// matrix instruction are cut off below the largest as if a subnormal's leading
// zeros were digits, and at the bottom of the mantissa 18732 even tokens cost
// an output 5e-4 of itself.
template <int D, int BITS>
__device__ __forceinline__ void value_operands(const uint32_t (&v)[2][4][Ring<D, BITS>::kValueWords], int i,
                                               v4u (&f)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {                // token pairs (0,1), (2,3) of each half
    const uint32_t* a = v[p / 2][2 * (p % 2)];
    const uint32_t* b = v[p / 2][2 * (p % 2) + 1];
    if constexpr (BITS == 4) {
      const uint32_t x =
          __builtin_amdgcn_perm(b[i / 8], a[i / 8], i % 8 ? 0x07060302u : 0x05040100u) ^ 0x88888888u;
      f[0][p] = x << 6 & 0x03C003C0u;
      f[1][p] = x << 2 & 0x03C003C0u;
      f[2][p] = x >> 2 & 0x03C003C0u;
      f[3][p] = x >> 6 & 0x03C003C0u;
    } else {
      const uint32_t x = a[i / 4] ^ 0x80808080u, y = b[i / 4] ^ 0x80808080u;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e][p] = __builtin_amdgcn_perm(y, x, 0x0C040C00u + (uint32_t)e * 0x00010001u);
    }
  }
}

template <int D, int BITS, int QT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4 * kv_decode_wgs(D, QT, WAVES))
void kv_decode_kernel(KvAttn a, KvSplit sp) {
  using R = Ring<D, BITS>;
  constexpr int E = D / 16;                    // elements of a lane's output tiles, and of a rotation lane
  constexpr int KM = D / 64;                   // matrix steps of a score
  constexpr int ROWS = 16 * QT;
  constexpr int PASS = E < 8 ? E : 8;   // elements of a row segment joined at once
  constexpr int PITCH = 16 * PASS + 4;
  constexpr int S = R::kStages, kStride = kStep * WAVES;
  constexpr int kNK = R::kLoads + 1, kNV = R::kLoads;    // direct loads of a step's keys (and scales), and values
  constexpr int QROWS = 4 * QT;                // query rows that a wavefront prepares (the first four do)
  constexpr int QBYTES = QROWS * 2 * D < 1024 ? 1024 : QROWS * 2 * D;
  __shared__ __align__(16) union {
    char ring[WAVES][R::kBytes];
    float o[WAVES][16][PITCH];
  } sh;
  __shared__ __align__(16) char qbuf[4][QBYTES];       // the rows as loaded, then each as its two int8 planes
  __shared__ float qscale[ROWS];
  __shared__ float stat[WAVES][16][2];

  const int tid = threadIdx.x, lane = tid % 64, col = lane % 16, quad = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int h = blockIdx.y, log2p = a.c.page_log2;
  int b = blockIdx.z, unit, split, tile, c0, chunk = sp.chunk;
  KvSeq s;
  bool alone = sp.splits == 1;                         // the sequence's only unit writes the output itself
  if (sp.balance) {
    unit = blockIdx.x % sp.units;
    tile = blockIdx.x / sp.units;
    const KvUnits u = kv_units(a, sp, -1, unit);
    if (u.b < 0) return;
    b = u.b;
    split = unit - u.first;
    chunk = u.chunk;
    alone = u.n == 1;
    s = u.seq;
  } else {
    split = blockIdx.x % sp.splits;
    tile = blockIdx.x / sp.splits;
    unit = b * sp.splits + split;
  }
  c0 = split * chunk;

  // The page numbers of the wavefront's next 64 steps, one a lane (two groups of 16 tokens a step), without waiting
  // for the sequence's length.
  int pages[2];
  auto find_pages = [&](int step) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t i = (c0 + kStep * wave + kStride * (step + lane) + 16 * u) >> log2p;
      const int p = i < a.width ? a.table[b * a.width + i] : -1;
      pages[u] = p < a.c.pages ? p : -1;
    }
  };
  find_pages(0);
  if (!sp.balance) s = kv_sequence(a, b);
  const int rows = s.n * a.group - tile * ROWS;      // valid rows from this tile on
  if (rows <= 0) return;
  // the tokens that the tile's last and first row see
  const int last = a.causal ? s.kv - s.n + kv_query_of(a, tile * ROWS + (rows < ROWS ? rows : ROWS) - 1) + 1 : s.kv;
  const int first = a.causal ? s.kv - s.n + kv_query_of(a, tile * ROWS) + 1 : s.kv;
  const int c1 = last < c0 + chunk ? last : c0 + chunk;
  if (c1 <= c0 && split > 0) return;                 // the join leaves it out by the same rule

  // ---- direct loads: the query rows, then the first steps
  if (wave < 4) {
    const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr_t)qbuf[wave];
#pragma unroll
    for (int n = 0; n < QBYTES / 1024; ++n) {
      const int off = n * 1024 + lane * 16, lr = off / (2 * D);
      const int row = tile * ROWS + 16 * (lr / 4) + 4 * wave + lr % 4;
      const int i = kv_query_of(a, row), head = h * a.group + row - i * a.group;
      const bool in = lr < QROWS && i < s.n;
      dma16(a.q.p + (in ? (s.first + i) * a.q.token + head * a.q.head + off % (2 * D) / 2 : 0),
            __builtin_amdgcn_readfirstlane(to + n * 1024));
    }
  }
  // Token 4 r + quad of a group of 16 is the one whose score ends up in register r of the lanes of `quad`, so a value
  // read of register r covers 4 neighbouring rows.  The keys' codes are laid down in operand order, 16 bytes a lane.
  const int turned = 4 * (col % 4) + col / 4;          // token of the lane's key codes, and of its scale
  const uint32_t koff = R::kRow < 64 ? 0 : turned * R::kRow + quad * 16, voff = lane * 16;
  char* ring = sh.ring[wave];
  const uint32_t ring0 = (uint32_t)(uintptr_t)(lds_ptr_t)ring;
  uint32_t present = 0;                                // bits 2 stage + u: the group's page is there
  int64_t row0, row1;
  // first rows of a step's two groups (of page 0 where there is none)
  auto find_rows = [&](int step, int stage) {
    const int j = c0 + kStep * wave + kStride * step;
    const int p0 = __builtin_amdgcn_readlane(pages[0], step % 64);
    const int p1 = j + 16 < c1 ? __builtin_amdgcn_readlane(pages[1], step % 64) : -1;
    const int mask = (1 << log2p) - 1;
    row0 = (((int64_t)(p0 < 0 ? 0 : p0) * a.c.heads + h) << log2p) + (j & mask);
    row1 = (((int64_t)(p1 < 0 ? 0 : p1) * a.c.heads + h) << log2p) + (j + 16 & mask);
    present = (present & ~(3u << 2 * stage)) | ((p0 >= 0) | (p1 >= 0) << 1) << 2 * stage;
  };
  auto load_keys = [&](int64_t r0, int64_t r1, int stage) {   // of the groups with these first rows, and all scales
    const uint32_t to = __builtin_amdgcn_readfirstlane(ring0 + stage * R::kStage);
    if constexpr (R::kRow < 64) {
      dma16(a.c.kc + (lane < 32 ? r0 : r1) * R::kRow + lane % 32 * 16, to);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < R::kLoads / 2; ++m)
          dma16(a.c.kc + (u ? r1 : r0) * R::kRow + m * 64, koff, to + (u * (R::kLoads / 2) + m) * 1024);
    }
    dma4((lane < 32 ? a.c.ks : a.c.vs) + (lane & 16 ? r1 : r0) + turned, to + 2 * R::kHalf);
  };
  auto load_values = [&](int64_t r0, int64_t r1, int stage) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(ring0 + stage * R::kStage + R::kHalf);
    if constexpr (R::kRow < 64) {
      dma16(a.c.vc + (lane < 32 ? r0 : r1) * R::kRow + lane % 32 * 16, to);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < R::kLoads / 2; ++m)
          dma16(a.c.vc + (u ? r1 : r0) * R::kRow + m * 1024, voff, to + (u * (R::kLoads / 2) + m) * 1024);
    }
  };
  int j0 = c0 + kStep * wave, step = 0, stage = 0;
#pragma unroll
  for (int n = 0; n < S; ++n)
    if (j0 + n * kStride < c1) {
      find_rows(n, n);
      load_keys(row0, row1, n);
      load_values(row0, row1, n);
    }

  // ---- the rotated queries, as two int8 planes, while the first steps arrive
  if (wave < 4) {
    if (S == 2 && j0 + kStride < c1) wait_vmcnt<2 * (kNK + kNV)>();
    else if (j0 < c1) wait_vmcnt<kNK + kNV>();
    else wait_vmcnt<0>();
    compiler_fence();
    const int r = tid / 16, seg = tid % 16;            // 16 rows, E elements a lane
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      char* mine = qbuf[wave] + (4 * t + r % 4) * 2 * D;
      const int i = kv_query_of(a, tile * ROWS + 16 * t + r);
      float x[E];
      load_row<E>(reinterpret_cast<const uint16_t*>(mine) + seg * E, a.bf16, x);
      if (i >= s.n) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.0f;
      }
      rotate_row<D>(x, seg);
      float top = 0.0f;
      bool fine = true;
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[e])), fine = fine & (fabsf(x[e]) < INFINITY);
      top = warp_max16(top);
      const float to = top > 0.0f ? 32512.0f / top : 0.0f;
      wave_lds_sync();                                 // the row's lanes have read it
      // n = 256 hi + lo with lo in [-128, 127]: lo is the low byte of n, hi the second of n + 128
      uint32_t n[E];
#pragma unroll
      for (int e = 0; e < E; ++e) n[e] = (uint32_t)(int)rintf(x[e] * to);
      auto bytes = [](uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3, uint32_t sel) {   // one byte of each
        return __builtin_amdgcn_perm(b1, b0, sel) | __builtin_amdgcn_perm(b3, b2, sel) << 16;
      };
#pragma unroll
      for (int e = 0; e < E; e += BITS == 4 ? 8 : 4) {   // neighbours in the operand: every second element of 8, or 4
#pragma unroll
        for (int par = 0; par < (BITS == 4 ? 2 : 1); ++par) {
          constexpr int step = BITS == 4 ? 2 : 1;
          // a lane of 4 elements (D = 64) holds half of such an 8
          if constexpr (BITS == 4 && E == 4) {
            const int at = query_place<D, BITS>(seg * E + par);
            *reinterpret_cast<uint16_t*>(mine + at) = (uint16_t)__builtin_amdgcn_perm(n[par + 2] + 128, n[par] + 128, 0x0C0C0501u);
            *reinterpret_cast<uint16_t*>(mine + D + at) = (uint16_t)__builtin_amdgcn_perm(n[par + 2], n[par], 0x0C0C0400u);
          } else {
            const int at = query_place<D, BITS>(seg * E + e + par);
            const uint32_t* m = n + e + par;
            *reinterpret_cast<uint32_t*>(mine + at) =
                bytes(m[0] + 128, m[step] + 128, m[2 * step] + 128, m[3 * step] + 128, 0x0C0C0501u);
            *reinterpret_cast<uint32_t*>(mine + D + at) = bytes(m[0], m[step], m[2 * step], m[3 * step], 0x0C0C0400u);
          }
        }
      }
      // sm_scale, the rotation's 1 / sqrt(D), the fixed point and the codes' 16
      const float f = a.scale * kv_rsqrt(D) * 1.44269504088896340736f * (top / 32512.0f) * (BITS == 4 ? 0.0625f : 1.0f);
      const uint64_t bad = __ballot(!fine);
      if (seg == 0) qscale[16 * t + r] = (bad >> (lane & 48)) & 0xFFFFu ? __uint_as_float(0x7FC00000u) : f;
    }
  }
  lds_barrier();
  v4i q[QT][2][KM];
  float qf[QT];
  int end[QT];                                        // tokens this lane's row sees
#pragma unroll
  for (int t = 0; t < QT; ++t) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int m = 0; m < KM; ++m)
        q[t][p][m] = *reinterpret_cast<const v4i*>(qbuf[col / 4] + (4 * t + col % 4) * 2 * D + p * D + quad * (D / 4) + 16 * m);
    qf[t] = qscale[16 * t + col];
    const int i = kv_query_of(a, tile * ROWS + 16 * t + col);
    end[t] = i >= s.n ? 0 : a.causal ? s.kv - s.n + i + 1 : s.kv;
  }

  v4f o[QT][E];
  const bool fine = !a.bf16;                           // fp16 outputs: the weights' rounding takes a second product
  v4f weight[QT];                                      // sum of the rounded weights (four times the same)
  float base[QT], l[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    base[t] = kUnset;
    l[t] = 0.0f;
    weight[t] = (v4f){0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i) o[t][i] = (v4f){0, 0, 0, 0};
  }

  // Direct loads return in order: waiting for a half leaves in flight what was issued after it.
  for (; j0 < c1; j0 += kStride, ++step, stage = S == 1 ? 0 : stage ^ 1) {
    const bool more = j0 + kStride < c1, refill = j0 + S * kStride < c1;
    const char* here_k = ring + stage * R::kStage;
    const char* here_v = here_k + R::kHalf;
    const char* here_s = here_v + R::kHalf;
    if (S == 2 && more) wait_vmcnt<2 * kNV + kNK>();
    else wait_vmcnt<kNV>();
    compiler_fence();
    uint32_t kw[2][R::kKeyWords];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (R::kRow < 64) {
        const v2u x = *reinterpret_cast<const v2u*>(here_k + (16 * u + turned) * R::kRow + quad * 8);
        kw[u][0] = x[0], kw[u][1] = x[1];
      } else {
#pragma unroll
        for (int m = 0; m < R::kLoads / 2; ++m) {
          const v4u x = *reinterpret_cast<const v4u*>(here_k + (u * (R::kLoads / 2) + m) * 1024 + lane * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) kw[u][4 * m + i] = x[i];
        }
      }
    }
    v4f ks[2], vs[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ks[u] = *reinterpret_cast<const v4f*>(here_s + 64 * u + 16 * quad);
      vs[u] = *reinterpret_cast<const v4f*>(here_s + 128 + 64 * u + 16 * quad);
    }
    const bool here[2] = {(present >> 2 * stage & 1) != 0, (present >> 2 * stage & 2) != 0};   // false past c1 too
    const bool whole = j0 + kStep <= first && here[0] && here[1];
    // ---- scores; the next keys load as soon as these are used
    v4i sc[QT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      v4i lo[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) sc[t][u] = lo[t] = (v4i){0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KM; ++k) {
        const v4i c = key_operand<D, BITS>(kw[u], k);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          sc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(c, q[t][0][k], sc[t][u], 0, 0, 0);
          lo[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(c, q[t][1][k], lo[t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) sc[t][u][r] = (sc[t][u][r] << 8) + lo[t][r];
    }
    if (refill) {
      if ((step + S) % 64 == 0) {
        find_pages(step + S);
#pragma unroll
        for (int t = 0; t < QT; ++t) {                   // the values' offset comes off
#pragma unroll
          for (int i = 0; i < E; ++i) o[t][i] += weight[t][0] * (BITS == 4 ? -0x1p-15f : -0x1p-17f);
          weight[t] = (v4f){0, 0, 0, 0};
        }
      }
      find_rows(step + S, stage);
      __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0): the reads are done
      load_keys(row0, row1, stage);
    }

    // ---- weights
    auto seen = [&](int t, int u, int r) { return (16 * u + 4 * r < end[t] - j0 - quad) & here[u]; };
    v8h w[QT], left_over[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float x[8], sum;
      for (bool again = false;; again = true) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          p[e] = __builtin_amdgcn_exp2f(__fmaf_rn((float)sc[t][e / 4][e % 4], ks[e / 4][e % 4] * qf[t], base[t]));
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = seen(t, e / 4, e % 4) ? p[e] : 0.0f;
        }
        sum = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = p[e] * vs[e / 4][e % 4];
        // a scale of NaN shows in the rows that see it, however small their weight, and in no others
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = seen(t, e / 4, e % 4) ? x[e] : 0.0f;
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
        // raise the maximum (rare); a row that has seen no token has an infinite sum
        if (again || !__any((top > kMostWeight) | (sum > kMostSum))) break;
        float best;
        for (bool shrunk = false;; shrunk = true) {
          best = kLowest;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int u = e / 4, r = e % 4;
            const float z = (float)sc[t][u][r] * (ks[u][r] * qf[t]) + __builtin_amdgcn_logf(fmaxf(vs[u][r], kLeastScale));
            best = fmaxf(best, (whole | seen(t, u, r)) ? z : kLowest);
          }
          best = max16_32(best);
          if (shrunk || !kv_shrink(best, base[t], qf[t], 0.0f)) break;
        }
        const float by = kv_raise(best, base[t]);
        l[t] *= by;
        weight[t] *= by;
#pragma unroll
        for (int i = 0; i < E; ++i) o[t][i] *= by;
      }
      l[t] += sum;
      v4u packed;
#pragma unroll
      for (int e = 0; e < 4; ++e) packed[e] = pack_f16x2_rn(x[2 * e], x[2 * e + 1]);
      w[t] = __builtin_bit_cast(v8h, packed);
      if (fine) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          packed[e] = pack_f16x2_rn(x[2 * e] - (float)w[t][2 * e], x[2 * e + 1] - (float)w[t][2 * e + 1]);
        left_over[t] = __builtin_bit_cast(v8h, packed);
      }
    }

    // ---- outputs; then the next values load
    if (refill) wait_vmcnt<(S - 1) * (kNK + kNV) + kNK>();
    else if (S == 2 && more) wait_vmcnt<kNK + kNV>();
    else wait_vmcnt<0>();
    compiler_fence();
    uint32_t vw[2][4][R::kValueWords];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const char* p = here_v + (16 * u + 4 * r + quad) * R::kRow + col * (R::kRow / 16);
        if constexpr (R::kRow < 64) vw[u][r][0] = *reinterpret_cast<const uint16_t*>(p);
        else if constexpr (R::kRow == 64) vw[u][r][0] = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (R::kRow == 128) {
          const v2u x = *reinterpret_cast<const v2u*>(p);
          vw[u][r][0] = x[0], vw[u][r][1] = x[1];
        } else {
          const v4u x = *reinterpret_cast<const v4u*>(p);
#pragma unroll
          for (int i = 0; i < 4; ++i) vw[u][r][i] = x[i];
        }
      }
    const v8h ones = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      weight[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, w[t], weight[t], 0, 0, 0);
      if (fine) weight[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, left_over[t], weight[t], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      v4u f[4];
      value_operands<D, BITS>(vw, i, f);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int t = 0; t < QT; ++t)
          o[t][i + n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, f[n]), w[t], o[t][i + n], 0, 0, 0);
      if (fine) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int t = 0; t < QT; ++t)
            o[t][i + n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, f[n]), left_over[t], o[t][i + n], 0, 0, 0);
      }
    }
    if (refill) {
      __builtin_amdgcn_s_waitcnt(0xC07F);
      load_values(row0, row1, stage);
    }
  }

  // ---- join the wavefronts, 16 rows at a time
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    l[t] = sum16_32(l[t]);
    const float most = kv_maximum(base[t], qf[t], qscale[16 * t + col]);
    __syncthreads();
    if (quad == 0) {
      stat[wave][col][0] = most;
      stat[wave][col][1] = l[t];
    }
    __syncthreads();
    float top = kLowest;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) top = fmaxf(top, stat[v][col][0]);
    const float mine = __builtin_amdgcn_exp2f(most - top);
    const float offset = weight[t][0] * (BITS == 4 ? -8.0f : -128.0f);
    const int r = tid / 16 % 16, seg = tid % 16;       // the first four wavefronts finish the rows
    float rtop = kLowest, sum = 0.0f, out[E];
#pragma unroll
    for (int v = 0; v < WAVES; ++v) rtop = fmaxf(rtop, stat[v][r][0]);
#pragma unroll
    for (int v = 0; v < WAVES; ++v) sum += __builtin_amdgcn_exp2f(stat[v][r][0] - rtop) * stat[v][r][1];
#pragma unroll
    for (int p = 0; p < E / PASS; ++p) {
      if (p) __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < PASS; ++i)
          sh.o[wave][col][PASS * (4 * quad + e) + i] =
              __fmaf_rn(o[t][PASS * p + i][e], BITS == 4 ? 0x1p18f : 0x1p24f, offset) * mine;
      __syncthreads();
      // four wavefronts sum four; with more, each group of four its own, and then the first four the groups
      const int g = wave / 4;
      v4f z[PASS / 4];
#pragma unroll
      for (int i = 0; i < PASS / 4; ++i) {
        z[i] = (v4f){0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < 4; ++v) z[i] += *reinterpret_cast<const v4f*>(&sh.o[4 * g + v][r][PASS * seg + 4 * i]);
      }
      if constexpr (WAVES > 4) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PASS / 4; ++i) *reinterpret_cast<v4f*>(&sh.o[g][r][PASS * seg + 4 * i]) = z[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PASS / 4; ++i)
#pragma unroll
          for (int v = 1; v < WAVES / 4; ++v) z[i] += *reinterpret_cast<const v4f*>(&sh.o[v][r][PASS * seg + 4 * i]);
      }
#pragma unroll
      for (int i = 0; i < PASS; ++i) out[PASS * p + i] = z[i / 4][i % 4];
    }
    if (wave >= 4) continue;
    const int rr = 16 * t + r;
    if (!alone) {
      if (rr < rows) {
        const int64_t at = sp.row(h, tile, unit, rr);
        float* dst = sp.o + at * D + seg * E;
#pragma unroll
        for (int i = 0; i < E; i += 4) *reinterpret_cast<v4f*>(dst + i) = (v4f){out[i], out[i + 1], out[i + 2], out[i + 3]};
        if (seg == 0) {
          sp.ml[2 * at] = rtop;
          sp.ml[2 * at + 1] = sum;
        }
      }
    } else {
      const float by = sum == 0.0f ? 0.0f : kv_rsqrt(D) / sum;
#pragma unroll
      for (int i = 0; i < E; ++i) out[i] = sum == 0.0f ? 0.0f : out[i] * by;
      rotate_row<D>(out, seg);
      if (rr < rows) {
        const int row = tile * ROWS + rr, i = kv_query_of(a, row), head = h * a.group + row - i * a.group;
        store_row<E>(a.o + ((s.first + i) * a.q_heads + head) * D + seg * E, a.bf16, out);
      }
    }
  }
}

// Joins the splits of each row: SEGS segments of 16 lanes take the splits in
// turn, E elements a lane, 16 splits of a segment at a time (their maxima and
// sums a lane each, so that the partial rows load without waiting for one
// another); the four segments of a wavefront are summed by lane swaps, the
// wavefronts through LDS, and the row is rotated back.  What counts is the
// chain of loads, not the bytes: 4, 16 or 64 segments, so that a segment has
// few splits; one where the rows alone fill the card.  Measured (join and what
// it joins, us): 6 splits of 1024 rows 20.7 with 4 segments, 21.6 with 16,
// 27.0 with 64; 16 splits of 64 rows 12.2, 11.6, 12.2; 128 splits of 32 rows
// 20.8 with 16, 19.7 with 64; 5 splits of 50000 rows 125 with one segment,
// 135 with 4.
template <int D, int SEGS>
__global__ __launch_bounds__(SEGS == 64 ? 1024 : 256) void kv_join_kernel(KvAttn a, KvSplit sp) {
  constexpr int E = D / 16, WAVES = SEGS < 4 ? 1 : SEGS / 4;   // wavefronts of a row
  constexpr int PER = SEGS == 64 ? 1 : 16 / SEGS;      // rows of a workgroup
  __shared__ __align__(16) float part[WAVES][D];
  __shared__ float stat[WAVES][2];
  const int sub = threadIdx.x / 16 % SEGS, seg = threadIdx.x % 16, h = blockIdx.y, b = blockIdx.z;
  const int row = blockIdx.x * PER + threadIdx.x / 16 / SEGS % PER;   // of the sequence's with this key head
  const int tile = row / sp.rows, rr = row - tile * sp.rows;
  int first = b * sp.splits, n = sp.splits, chunk = sp.chunk;
  KvSeq s;
  if (sp.balance) {
    const KvUnits u = kv_units(a, sp, b, 0);           // takes all 64 lanes: before any returns
    first = u.first, n = u.n, chunk = u.chunk, s = u.seq;
    if (n == 1) return;                                // written by its only unit
  }
  // With SEGS = 1 a wavefront has four rows, of which some may end here and below; from here on lanes of one row
  // meet only, and with more segments a wavefront, or all that meet, has one row.
  if (tile >= sp.tiles || rr >= sp.kept) return;
  // the first 16 splits' maxima and sums, without waiting for the sequence's lengths
  const int64_t at = sp.row(h, tile, first, rr);
  int z = sub + seg * SEGS;                            // this lane's split
  float mz = kLowest, lz = 0.0f;
  if (z < n) {
    mz = sp.ml[2 * (at + (int64_t)z * sp.kept)];
    lz = sp.ml[2 * (at + (int64_t)z * sp.kept) + 1];
  }
  if (!sp.balance) s = kv_sequence(a, b);
  const int i = kv_query_of(a, row);
  if (i >= s.n) return;
  // the splits that the row's tile ran: up to the last token its last row sees
  int last = s.kv;
  if (a.causal) {
    int r1 = (tile + 1) * sp.rows - 1;
    r1 = r1 < s.n * a.group ? r1 : s.n * a.group - 1;
    last = s.kv - s.n + kv_query_of(a, r1) + 1;
  }
  const int ran = last > 0 ? (last - 1) / chunk + 1 : 1;
  n = ran < n ? ran : n;
  float m = kLowest, l = 0.0f, x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.0f;
  for (int z0 = sub; z0 < n; z0 += 16 * SEGS) {
    if (z0 != sub) {
      z = z0 + seg * SEGS;
      if (z < n) {
        mz = sp.ml[2 * (at + (int64_t)z * sp.kept)];
        lz = sp.ml[2 * (at + (int64_t)z * sp.kept) + 1];
      }
    }
    mz = z < n ? mz : kLowest;
    lz = z < n ? lz : 0.0f;
    const float next = fmaxf(m, warp_max16(mz)), keep = __builtin_amdgcn_exp2f(m - next);
    const float w = z < n ? __builtin_amdgcn_exp2f(mz - next) : 0.0f;
    m = next;
    l = l * keep + lz * w;                             // summed over the lanes below
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= keep;
    const int count = (n - z0 + SEGS - 1) / SEGS;
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      if (k >= count) break;
      const float wk = __shfl(w, k, 16);
      const float* o = sp.o + (at + (int64_t)(z0 + k * SEGS) * sp.kept) * D + seg * E;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const v4f y = *reinterpret_cast<const v4f*>(o + e);
#pragma unroll
        for (int g = 0; g < 4; ++g) x[e + g] += y[g] * wk;
      }
    }
  }
#pragma unroll
  for (int k = 1; k < 16; k <<= 1) l += __shfl_xor(l, k);
  float sum = l;
  if constexpr (SEGS > 1) {
    const float top = max16_32(m), by = __builtin_amdgcn_exp2f(m - top);
    sum = sum16_32(l * by);
    m = top;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = sum16_32(x[e] * by);
  }
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x / 64;
    if (sub % 4 == 0) {
      if (seg == 0) {
        stat[wave][0] = m;
        stat[wave][1] = sum;
      }
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<v4f*>(&part[wave][seg * E + e]) = (v4f){x[e], x[e + 1], x[e + 2], x[e + 3]};
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) m = fmaxf(m, stat[v][0]);
    sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; v += 4) {
      const float by = __builtin_amdgcn_exp2f(stat[v + sub][0] - m);
      sum += stat[v + sub][1] * by;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const v4f y = *reinterpret_cast<const v4f*>(&part[v + sub][seg * E + e]);
#pragma unroll
        for (int g = 0; g < 4; ++g) x[e + g] += y[g] * by;
      }
    }
    sum = sum16_32(sum);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = sum16_32(x[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = sum == 0.0f ? 0.0f : x[e] * (kv_rsqrt(D) / sum);
  rotate_row<D>(x, seg);
  if (sub % 4 == 0) store_row<E>(a.o + ((s.first + i) * a.q_heads + h * a.group + row - i * a.group) * D + seg * E, a.bf16, x);
}

template <int D, int BITS, int QT, int WAVES>
hipError_t run(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  KvSplit sp = p.split;
  sp.o = static_cast<float*>(workspace);
  sp.ml = sp.o ? sp.o + p.parts * D : nullptr;
  const dim3 grid(sp.balance ? sp.units * sp.tiles : sp.splits * sp.tiles, a.c.heads, sp.balance ? 1 : a.batch);
  kv_decode_kernel<D, BITS, QT, WAVES><<<grid, 64 * WAVES, 0, stream>>>(a, sp);
  if (hipError_t e = hipGetLastError()) return e;
  return sp.splits > 1 ? launch_kv_join(a, sp, stream) : hipSuccess;
}

template <int D, int BITS>
hipError_t run(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  if (p.waves > 4) return run<D, BITS, 1, kv_decode_wide(D)>(a, p, workspace, stream);
  return p.split.rows == 16 ? run<D, BITS, 1, 4>(a, p, workspace, stream) : run<D, BITS, 2, 4>(a, p, workspace, stream);
}

}  // namespace

// A call runs in one of three ways, by `base`, its workgroups when each takes
// a whole sequence for one key head and tile of rows, and by `slots`, the
// workgroups that 256 CUs hold.  Measured with heads of 128 in 4 bits, 8 key
// heads of 4 query heads (slots 1024), us:
//   one workgroup of 4 wavefronts each, no join: while the walk is short
//   against starting, splitting and joining, and where it fills the card;
//   one workgroup of 16 wavefronts (8 for heads of 256) each, at most one a
//   CU, no join: longer walks that about fill the CUs, and short ones that
//   would leave most idle (there the split is as fast in a captured graph, but
//   its second launch costs a stream of single calls 4 us);
//   units of equal work over all sequences, then the join: the rest.  The
//   units fill the card once: twice as many cost 51 us, four times as many
//   58 us, against 45 us for 32 sequences of up to 8192 tokens.
//     base  tokens   4 waves  16 waves  split
//        8     512       8.9       9.9   10.8
//        8    1024      12.3      12.1   10.8 (single calls: 13.5, 13.6, 17.5)
//        8    2048      19.3      15.5   11.2
//      128    2048      20.4      16.8   19.1
//      128    4096      34.3      23.3   23.6 (unequal lengths: 34.0, 23.1, 20.6)
//      256    1024      13.8      16.1   18.8
//      256    4096      34.5      28.7   34.0 (unequal lengths: 33.6, 25.0, 28.8)
//      512    4096      58.1      61.8   66.0 (unequal lengths: 47.6, 48.6, 52.8)
//     1024    1024      29.1      52.5   34.0
//     6000    2048       291       ---    301 (unequal lengths: 196, ---, 226)
// More sequences than kv_units counts take equal chunks instead: 300 sequences
// of up to 8192 tokens and one key head, 58.7 us in chunks of 2048 against
// 68.0 whole; where base fills the card (8 key heads, up to 16384 tokens) 660
// whole, 719 in chunks of 4096, 750 in chunks of 2048.
KvPlan kv_decode_plan(const KvAttn& a) {
  KvPlan p{};
  const int64_t rows = (int64_t)a.max_q * a.group;
  KvSplit& s = p.split;
  s.rows = rows <= 16 ? 16 : 32;
  s.tiles = (int)((rows + s.rows - 1) / s.rows);
  s.kept = (int)(rows < s.rows ? rows : s.rows);
  p.waves = 4;
  s.splits = 1;
  s.chunk = a.max_kv < 128 ? 128 : (a.max_kv + 127) / 128 * 128;
  s.units = a.batch;
  const int64_t heads = (int64_t)s.tiles * a.c.heads, base = heads * a.batch;
  const int64_t slots = 256 * kv_decode_wgs(a.c.head_dim, s.rows / 16, 4);   // resident on 256 CUs
  if (a.max_kv <= 512 || (a.max_kv <= 1024 && 4 * base >= slots) || (a.max_kv <= 4096 && 2 * base >= slots) ||
      (a.max_kv <= 8192 && base >= 4 * slots))
    return p;
  if (s.rows == 16 && base <= 256 && a.max_kv <= (base < 128 ? 1024 : 16 * base)) {
    p.waves = kv_decode_wide(a.c.head_dim);
    return p;
  }
  if (a.batch <= 256) {
    const int64_t want = slots / heads;
    s.balance = (int)(want < a.batch ? a.batch : want);
    s.by_balance = kv_divider((uint32_t)s.balance);
    s.units = 2 * (int64_t)a.batch <= s.balance ? s.balance : s.balance + a.batch;
    const int64_t most = (int64_t)a.batch * ((a.max_kv + 255) / 256);   // chunks have 256 tokens at least
    if (s.units > most) s.units = (int)most;
    s.splits = (a.max_kv + 255) / 256;                                  // a sequence's units at most
    if (s.splits > s.units) s.splits = s.units;
  } else {
    const int chunk = base < slots ? 2048 : 16384;
    if (a.max_kv <= 2 * chunk) return p;
    s.chunk = chunk;
    s.splits = (a.max_kv + s.chunk - 1) / s.chunk;
    s.units = a.batch * s.splits;
  }
  p.parts = heads * s.units * s.kept;
  p.bytes = (size_t)p.parts * (a.c.head_dim + 2) * 4;
  return p;
}

namespace {

template <int D>
hipError_t join(const KvAttn& a, const KvSplit& sp, hipStream_t stream) {
  const unsigned rows = (unsigned)a.max_q * a.group;
  const int64_t all = (int64_t)rows * a.c.heads * a.batch;
  if (sp.splits <= 16 && all >= 16384) kv_join_kernel<D, 1><<<dim3((rows + 15) / 16, a.c.heads, a.batch), 256, 0, stream>>>(a, sp);
  else if (sp.splits <= 8) kv_join_kernel<D, 4><<<dim3((rows + 3) / 4, a.c.heads, a.batch), 256, 0, stream>>>(a, sp);
  else if (sp.splits <= 32) kv_join_kernel<D, 16><<<dim3(rows, a.c.heads, a.batch), 256, 0, stream>>>(a, sp);
  else kv_join_kernel<D, 64><<<dim3(rows, a.c.heads, a.batch), 1024, 0, stream>>>(a, sp);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_join(const KvAttn& a, const KvSplit& sp, hipStream_t stream) {
  return a.c.head_dim == 64 ? join<64>(a, sp, stream)
         : a.c.head_dim == 128 ? join<128>(a, sp, stream) : join<256>(a, sp, stream);
}

hipError_t launch_kv_decode(const KvAttn& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  switch (a.c.head_dim * 16 + a.c.bits) {
    case 64 * 16 + 4: return run<64, 4>(a, p, workspace, stream);
    case 64 * 16 + 8: return run<64, 8>(a, p, workspace, stream);
    case 128 * 16 + 4: return run<128, 4>(a, p, workspace, stream);
    case 128 * 16 + 8: return run<128, 8>(a, p, workspace, stream);
    case 256 * 16 + 4: return run<256, 4>(a, p, workspace, stream);
    default: return run<256, 8>(a, p, workspace, stream);
  }
}

}  // namespace convrot
