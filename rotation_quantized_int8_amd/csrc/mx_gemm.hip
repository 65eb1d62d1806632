// The product of microscaled 4-bit rows, Y = out(X W^T + bias + residual), on
// the scaled matrix instructions of gfx950.
//
// Mathematics.  v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 rows by 32 rows
// over 64 elements, two blocks of 32 with a scale each: a lane holds one block of
// one row (16 bytes) and, in a byte of a register, its scale.  The sum over K does
// not ask which blocks an instruction takes, as long as both operands agree: of a
// rotation group (8 blocks, 128 bytes a row) lane half q takes blocks 4q .. 4q + 3,
// one an instruction, so that its four scales are one word of the layout
// [K / 256, rows, 8].  Of the two shapes this one is faster (operands in registers:
// 9.0 PFLOP/s against 4.8 with 16x16x128; with operands of random bits 6.6 against
// 4.6, where the clock gives way).
//
// Data flow.  Tiles as in the int8 product: direct global->LDS loads into a ring
// of STAGES slices of one rotation group, 16-byte chunks XOR-swizzled by
// (row >> 1) & 7 (16 rows cover all banks; row & 7 leaves 7 times the conflicts);
// the slice's scales, 8 bytes a row, follow the codes in the same ring.  The weight tile is the left operand, so a lane's
// accumulators are fours of neighbouring outputs of one row.
//
// Bound and measured (us, one call after another in a graph, operands in turn; a call
// traced alone takes 0.5 to 1 more).  Large: 8192^3 254 to 270 (4.1 to 4.3 PFLOP/s)
// in tiles of 256x256, the matrix cores busy 53 % of the cycles at the 1.8 GHz that
// the card holds under it, the rest waits of wavefronts that enter and leave a slice
// together.  Middle: 1024 x 2048 x 8192 18.7, with bias and residual 21.4: 256
// workgroups put one wavefront on a SIMD, whose barrier, LDS reads and products stand
// in line (matrix cores 13 % busy).  Small: 777 x 1003 x 768 4.3, 24 x 8192 x 2048 4.5,
// a launch, a round trip for the first slice and 0.25 a slice.  1 x 2048 x 2048 with
// its quantisation 3.5.
//
// Rows past M or N repeat the last valid row for the loads and are dropped in
// the epilogue.

#include <type_traits>

#include "dma.hpp"
#include "mx.hpp"

namespace convrot {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// The four registers of e2m1 operands in the eight that the builtins take.
__device__ __forceinline__ v8i as_operand(v4i v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// acc += (w 2^sw) (x 2^sx)^T; byte kk of the registers sw and sx (4: e2m1).
template <int kk>
__device__ __forceinline__ v4f mx_mfma(v4i w, v4i x, v4f acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(as_operand(w), as_operand(x), acc, 4, 4, kk, sw, kk, sx);
}
template <int kk>
__device__ __forceinline__ v16f mx_mfma(v4i w, v4i x, v16f acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(as_operand(w), as_operand(x), acc, 4, 4, kk, sw, kk, sx);
}

__device__ __forceinline__ float in16_to_f32(uint16_t bits, int bf16) {
  return bf16 ? bf16_to_f32(bits) : __half2float(__ushort_as_half(bits));
}

// Two finished sums to the output's type, each rounded once to nearest even.
__device__ __forceinline__ uint32_t out_pair(float a, float b, int bf16) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return bf16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2)) : pack_f16x2_rn(a, b);
}

// C neighbouring outputs of row m from column n: y + bias + residual in fp32,
// rounded once and stored.  `whole`: all C columns are inside (rows may start at
// any element); else element by element.  The residual is read by the thread that
// writes the element, before it: it may be the output.
template <int C>
__device__ __forceinline__ void finish(const MxGemm& p, float (&y)[C], int64_t m, int64_t n, const float (&bias)[C],
                                       bool whole) {
  typedef uint16_t vec __attribute__((ext_vector_type(C)));
  typedef vec vec_any __attribute__((aligned(2)));
  const int64_t at = m * p.N + n;
  const uint16_t* res = static_cast<const uint16_t*>(p.res);
  uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
  for (int r = 0; r < C; ++r) y[r] += bias[r];
  if (res) {
    vec h;
    if (whole) {
      h = __builtin_nontemporal_load(reinterpret_cast<const vec_any*>(res + at));
    } else {
#pragma unroll
      for (int r = 0; r < C; ++r) h[r] = n + r < p.N ? res[at + r] : 0;
    }
#pragma unroll
    for (int r = 0; r < C; ++r) y[r] += in16_to_f32(h[r], p.bf16);
  }
  vec v;
#pragma unroll
  for (int r = 0; r < C; r += 2) {
    const uint32_t w = out_pair(y[r], y[r + 1], p.bf16);
    v[r] = (uint16_t)w;
    v[r + 1] = (uint16_t)(w >> 16);
  }
  if (whole) {
    __builtin_nontemporal_store(v, reinterpret_cast<vec_any*>(out + at));
  } else {
#pragma unroll
    for (int r = 0; r < C; ++r)
      if (n + r < p.N) out[at + r] = v[r];
  }
}

// -0, so that a sum without a bias stays as it is.
template <int C>
__device__ __forceinline__ void load_bias(const MxGemm& p, int64_t n, float (&bias)[C]) {
#pragma unroll
  for (int r = 0; r < C; ++r) bias[r] = p.bias ? p.bias[n + r < p.N ? n + r : p.N - 1] : -0.0f;
}

template <int WAVES_M, int WAVES_N, int FM, int FN, int STAGES>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N)
mx_gemm_kernel(MxGemm p) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = 32 * FM, WN = 32 * FN;
  constexpr int BM = WAVES_M * WM, BN = WAVES_N * WN;
  constexpr int NKK = 4;                                          // K steps (64 elements) of a slice
  constexpr int XL = BM / 8 / NW, WL = BN / 8 / NW;               // 1 KiB blocks (8 rows) a wave loads per slice
  constexpr int SL = ((BM + BN) / 32 + NW - 1) / NW;              // 256-byte blocks of scales (32 rows)
  constexpr int LPW = XL + WL + SL;
  constexpr int XBYTES = BM * 128, WBYTES = BN * 128, SBYTES = SL * NW * 256;
  constexpr int STAGE = XBYTES + WBYTES + SBYTES;
  constexpr int kAhead = (STAGES - 2) * LPW;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM % 32 == 0, "blocks split evenly over waves");
  static_assert(STAGES >= 2 && kAhead < 64, "pipeline depth");
  constexpr bool kDeep = FM * FN <= 4;                            // fragments of whole slices in registers

  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int64_t M = p.M, N = p.N, nk = p.K / kGroup, ld = p.K / 2;
  const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN, T = tiles_m * tiles_n;
  // XCD-aware order as in the int8 product (fewer than 2^23 tiles): the i-th
  // workgroup on XCD x takes the i-th tile of a contiguous range
  const uint32_t b = blockIdx.x, xcd = b & 7, per = (uint32_t)T >> 3, rem = (uint32_t)T & 7;
  const uint32_t t = xcd * per + (xcd < rem ? xcd : rem) + (b >> 3);
  const uint32_t gm = (uint32_t)p.group_m, in_group = gm * (uint32_t)tiles_n;
  const uint32_t group = t / in_group, in = t - group * in_group, first_m = group * gm;
  const uint32_t gsize = (uint32_t)tiles_m - first_m < gm ? (uint32_t)tiles_m - first_m : gm;
  const int64_t m0 = (int64_t)(first_m + in % gsize) * BM, n0 = (int64_t)(in / gsize) * BN;

  // Sources of this wave's loads: a base for the tile, which advances by slices,
  // and an offset for each lane (at most 256 rows of 64 KiB).
  uint32_t offx[XL], offw[WL], offs[SL];
  bool sc_x[SL];
  auto key = [](int r) { return (r >> 1) & 7; };   // swizzle of row r's chunks
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = 8 * (wave * XL + i) + (lane >> 3);
    const int64_t row = m0 + r < M ? m0 + r : M - 1;
    offx[i] = (uint32_t)((row - m0) * ld) + 16 * ((lane & 7) ^ key(r));
  }
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int r = 8 * (wave * WL + i) + (lane >> 3);
    const int64_t row = n0 + r < N ? n0 + r : N - 1;
    offw[i] = (uint32_t)((row - n0) * ld) + 16 * ((lane & 7) ^ key(r));
  }
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    // 32 rows a load, of one operand (past both tiles: weight rows that no one reads)
    const int r0 = 32 * (wave * SL + i), r = r0 + (lane >> 1);
    sc_x[i] = r0 < BM;
    const int64_t first = sc_x[i] ? m0 : n0, rows = sc_x[i] ? M : N;
    const int64_t row = first + (sc_x[i] ? r : r - BM);
    offs[i] = (uint32_t)(((row < rows ? row : rows - 1) - first) * 8) + 4 * (lane & 1);
  }
  const uint8_t* basex = p.x + m0 * ld;
  const uint8_t* basew = p.w + n0 * ld;
  const uint8_t* basexs = p.xs + m0 * 8;
  const uint8_t* basews = p.ws + n0 * 8;
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
  // load u of slice kt's LPW to the buffer at `at`
  auto issue_one = [&](int u, int64_t kt, uint32_t at) {
    if (u < XL) {
      dma16(basex + kt * 128, offx[u], __builtin_amdgcn_readfirstlane(at + (wave * XL + u) * 1024));
    } else if (u < XL + WL) {
      dma16(basew + kt * 128, offw[u - XL], __builtin_amdgcn_readfirstlane(at + XBYTES + (wave * WL + u - XL) * 1024));
    } else {
      const int i = u - XL - WL;
      dma4(sc_x[i] ? basexs + kt * M * 8 : basews + kt * N * 8, offs[i],
           __builtin_amdgcn_readfirstlane(at + XBYTES + WBYTES + (wave * SL + i) * 256));
    }
  };
  auto issue = [&](int64_t kt, int stage) {
#pragma unroll
    for (int u = 0; u < LPW; ++u) issue_one(u, kt, lds_base + stage * STAGE);
  };

  v16f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int frow = lane & 31, fq = lane >> 5;
  // Fragments of a K step (64 elements) of 32 rows; rows are 32 apart, so the
  // swizzle is the lane's own.
  const uint32_t lw = XBYTES + (wn * WN + frow) * 128, lx = (wm * WM + frow) * 128;
  uint32_t chunk[NKK];
#pragma unroll
  for (int kk = 0; kk < NKK; ++kk) chunk[kk] = 16u * ((NKK * fq + kk) ^ key(frow));
  const uint32_t lsw = XBYTES + WBYTES + (BM + wn * WN + frow) * 8 + NKK * fq;
  const uint32_t lsx = XBYTES + WBYTES + (wm * WM + frow) * 8 + NKK * fq;
  auto load_frags = [&](int kk, uint32_t st, v4i (&w)[FN], v4i (&x)[FM]) {
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = *reinterpret_cast<const v4i*>(smem + (st + lw + chunk[kk]) + i * 4096);
#pragma unroll
    for (int j = 0; j < FM; ++j) x[j] = *reinterpret_cast<const v4i*>(smem + (st + lx + chunk[kk]) + j * 4096);
  };
  auto load_scales = [&](uint32_t st, int (&w)[FN], int (&x)[FM]) {
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = *reinterpret_cast<const int*>(smem + (st + lsw) + i * 256);
#pragma unroll
    for (int j = 0; j < FM; ++j) x[j] = *reinterpret_cast<const int*>(smem + (st + lsx) + j * 256);
  };

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < nk) issue(s, s);
  if (nk >= STAGES - 1) wait_vmcnt<kAhead>();
  else wait_vmcnt<0>();
  lds_barrier();
  if (STAGES - 1 < nk) issue(STAGES - 1, STAGES - 1);
  int stage = 0;
  using yes = std::true_type;
  using no = std::false_type;
  int64_t kt = 0;
  if constexpr (kDeep) {
    // Small tiles: a step's products take less than an LDS read, so the fragments
    // of a whole slice are read under the products of the slice before it (128x64
    // tile, 1024 x 2048 x 8192 without bias: 18.4 us; step by step 21.3).  Behind the barrier every
    // read of slice kt is done and slice kt + 1 is published.
    struct Slice {
      v4i w[NKK][FN], x[NKK][FM];
      int sw[FN], sx[FM];
    } one, two;
    auto read = [&](Slice& s, uint32_t st) {
      load_scales(st, s.sw, s.sx);
#pragma unroll
      for (int kk = 0; kk < NKK; ++kk) load_frags(kk, st, s.w[kk], s.x[kk]);
    };
    auto products = [&](auto kk, const Slice& s) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
          acc[i][j] = mx_mfma<kk.value>(s.w[kk.value][i], s.x[kk.value][j], acc[i][j], s.sw[i], s.sx[j]);
    };
    auto all = [&](const Slice& s) {
      products(std::integral_constant<int, 0>{}, s);
      products(std::integral_constant<int, 1>{}, s);
      products(std::integral_constant<int, 2>{}, s);
      products(std::integral_constant<int, 3>{}, s);
    };
    auto slice = [&](int64_t kt, auto refill, const Slice& now, Slice& next) {
      const uint32_t st = stage * STAGE;
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      if constexpr (refill) wait_vmcnt<kAhead>();
      else wait_vmcnt<0>();
      lds_barrier();
      read(next, stage * STAGE);
      if constexpr (refill) {
#pragma unroll
        for (int u = 0; u < LPW; ++u) issue_one(u, kt + STAGES, lds_base + st);
      }
      all(now);
    };
    read(one, 0);
    for (; kt + 1 < nk - STAGES; kt += 2) {
      slice(kt, yes{}, one, two);
      slice(kt + 1, yes{}, two, one);
    }
    if (kt < nk - STAGES) {
      slice(kt, yes{}, one, two);
      ++kt;
      one = two;
    }
    for (; kt < nk - 1; ++kt) {
      slice(kt, no{}, one, two);
      one = two;
    }
    all(one);
  } else {
    // Large tiles: one slice in NKK steps, each step's fragments read under the
    // products of the one before.  Before the last step every read of the slice is
    // done, so behind one barrier the slice after it is published and its buffer
    // refilled, a few loads at a time between the products, and the next slice's
    // first fragments are read under the last step's products.
    v4i fw[2][FN], fx[2][FM];
    int sw[FN], sx[FM];
    auto products = [&](auto kk) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
          acc[i][j] = mx_mfma<kk.value>(fw[kk.value & 1][i], fx[kk.value & 1][j], acc[i][j], sw[i], sx[j]);
    };
    auto slice = [&](int64_t kt, auto refill, auto last) {
      const uint32_t st = stage * STAGE;
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      const uint32_t next = stage * STAGE;
      load_frags(1, st, fw[1], fx[1]);
      products(std::integral_constant<int, 0>{});
      load_frags(2, st, fw[0], fx[0]);
      products(std::integral_constant<int, 1>{});
      load_frags(3, st, fw[1], fx[1]);
      products(std::integral_constant<int, 2>{});
      int nsw[FN], nsx[FM];
      if constexpr (!last) {
        if constexpr (refill) wait_vmcnt<kAhead>();
        else wait_vmcnt<0>();
        lds_barrier();
        load_scales(next, nsw, nsx);
        load_frags(0, next, fw[0], fx[0]);
      }
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          constexpr int kProducts = FN * FM;
          const int t = i * FM + j;
          acc[i][j] = mx_mfma<NKK - 1>(fw[1][i], fx[1][j], acc[i][j], sw[i], sx[j]);
          if constexpr (refill) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = t * LPW / kProducts; u < (t + 1) * LPW / kProducts; ++u)
              issue_one(u, kt + STAGES, lds_base + st);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      if constexpr (!last) {
#pragma unroll
        for (int i = 0; i < FN; ++i) sw[i] = nsw[i];
#pragma unroll
        for (int j = 0; j < FM; ++j) sx[j] = nsx[j];
      }
    };
    load_scales(0, sw, sx);
    load_frags(0, 0, fw[0], fx[0]);
    for (; kt < nk - STAGES; ++kt) slice(kt, yes{}, no{});
    for (; kt < nk - 1; ++kt) slice(kt, no{}, no{});
    slice(kt, no{}, yes{});
  }

  // The finished tile goes through LDS as fp32, one fragment row of each wavefront
  // at a time and two buffers in turn, so that residual and output move in whole
  // 16-byte chunks of rows.  The ring is free behind the first barrier.
  constexpr int ROWB = BN * 4 + 16, ROWS = 32 * WAVES_M, BUF = ROWS * ROWB;
  static_assert((FM > 1 ? 2 : 1) * BUF <= STAGES * STAGE, "the staged rows must fit in the ring");
  constexpr int CPR = BN / 8, NTH = 64 * NW;   // 8 outputs a thread at a time
  static_assert(NTH % CPR == 0 && ROWS % (NTH / CPR) == 0, "a thread keeps its columns");
  const int cc = tid % CPR;
  const int64_t n = n0 + 8 * cc;
  float bias[8];
  load_bias(p, n, bias);
  const bool whole = n + 8 <= N;
  lds_barrier();
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    char* buf = smem + (j & 1) * BUF;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<v4f*>(buf + (wm * 32 + frow) * ROWB + (wn * WN + i * 32 + 8 * g + 4 * fq) * 4) =
            v4f{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    lds_barrier();
    if (n < N) {
#pragma unroll 2
      for (int r = tid / CPR; r < ROWS; r += NTH / CPR) {
        const int64_t m = m0 + (r >> 5) * WM + j * 32 + (r & 31);
        if (m >= M) continue;
        const v4f* src = reinterpret_cast<const v4f*>(buf + r * ROWB + cc * 32);
        const v4f a = src[0], c = src[1];
        float y[8] = {a[0], a[1], a[2], a[3], c[0], c[1], c[2], c[3]};
        finish<8>(p, y, m, n, bias, whole);
      }
    }
  }
}

// Few rows: a workgroup owns 16 weight rows (outputs) and all of up to 16 NB
// activation rows; its wavefronts take the rotation groups in turn, straight
// from memory to registers (each weight byte is read once on the whole card),
// and add their sums in LDS in the order of the wavefronts.
template <int NB, int WAVES>
__global__ void __launch_bounds__(64 * WAVES)
mx_few_kernel(MxGemm p) {
  __shared__ __align__(16) float part[WAVES][NB][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int frow = lane & 15, fq = lane >> 4;
  const int64_t M = p.M, N = p.N, G = p.K / kGroup, ld = p.K / 2;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t wrow = n0 + frow < N ? n0 + frow : N - 1;
  const uint8_t* w = p.w + wrow * ld + 32 * fq;
  const uint8_t* ws = p.ws + wrow * 8 + 2 * fq;
  const uint8_t* x[NB];
  const uint8_t* xs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t row = 16 * j + frow < M ? 16 * j + frow : M - 1;
    x[j] = p.x + row * ld + 32 * fq;
    xs[j] = p.xs + row * 8 + 2 * fq;
  }
  v4f acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = v4f{0, 0, 0, 0};
#pragma unroll 4
  for (int64_t g = wave; g < G; g += WAVES) {
    const v4i* pw = reinterpret_cast<const v4i*>(w + g * 128);
    const v4i w0 = __builtin_nontemporal_load(pw), w1 = __builtin_nontemporal_load(pw + 1);
    const int sw = *reinterpret_cast<const uint16_t*>(ws + g * N * 8);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const v4i* px = reinterpret_cast<const v4i*>(x[j] + g * 128);
      const v4i x0 = px[0], x1 = px[1];
      const int sx = *reinterpret_cast<const uint16_t*>(xs[j] + g * M * 8);
      acc[j] = mx_mfma<0>(w0, x0, acc[j], sw, sx);
      acc[j] = mx_mfma<1>(w1, x1, acc[j], sw, sx);
    }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) *reinterpret_cast<v4f*>(part[wave][j][lane]) = acc[j];
  __syncthreads();
  if (wave >= NB) return;
  const int j = wave;
  v4f y = *reinterpret_cast<const v4f*>(part[0][j][lane]);
#pragma unroll
  for (int v = 1; v < WAVES; ++v) y += *reinterpret_cast<const v4f*>(part[v][j][lane]);
  const int64_t m = 16 * j + frow, n = n0 + 4 * fq;
  if (m >= M || n >= N) return;
  float bias[4], z[4] = {y[0], y[1], y[2], y[3]};
  load_bias(p, n, bias);
  finish<4>(p, z, m, n, bias, n + 4 <= N);
}

// The whole linear for few short rows (M G <= 32 rotation groups, G <= 32): every
// workgroup quantises the activations itself, a group to 16 lanes, while its
// weights are on their way, then works as mx_few_kernel does, in the same order.
// One launch instead of two, and no workspace.
constexpr int kFusedWaves = 8, kFusedGroups = 4 * kFusedWaves;
template <bool kBF16>
__global__ void __launch_bounds__(64 * kFusedWaves)
mx_few_fused_kernel(MxGemm p, const uint16_t* __restrict__ X) {
  extern __shared__ __align__(16) char smem[];      // kFusedGroups slots; the sums of the wavefronts later
  __shared__ __align__(16) uint8_t codes[kFusedGroups * 128];
  __shared__ __align__(8) uint8_t scales[kFusedGroups * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int frow = lane & 15, fq = lane >> 4;
  const int M = (int)p.M, G = (int)(p.K / kGroup);
  const int64_t N = p.N, ld = p.K / 2, n0 = (int64_t)blockIdx.x * 16;
  const int64_t wrow = n0 + frow < N ? n0 + frow : N - 1;
  v4i w[4][2];
  int sw[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int g = wave + kFusedWaves * t;
    if (g >= G) break;
    const v4i* pw = reinterpret_cast<const v4i*>(p.w + wrow * ld + g * 128 + 32 * fq);
    w[t][0] = __builtin_nontemporal_load(pw);
    w[t][1] = __builtin_nontemporal_load(pw + 1);
    sw[t] = *reinterpret_cast<const uint16_t*>(p.ws + (g * N + wrow) * 8 + 2 * fq);
  }
  const int seg = threadIdx.x >> 4, sl = threadIdx.x & 15;
  if (seg < M * G) {
    // groups of a row lie side by side
    const v4i* px = reinterpret_cast<const v4i*>(X + (int64_t)seg * kGroup + 16 * sl);
    double y[16];
    rotate_loaded<kBF16>(px[0], px[1], smem + seg * kSlotBytes, sl, y);
    float f[16];
    mx_rotated<kBF16>(y, f);
    const int row = seg / G, g = seg - row * G;
    mx_store<mx_up(kBF16)>(f, row, M, p.K, g, sl, codes, scales);
  }
  __syncthreads();
  v4f acc = {0, 0, 0, 0};
  const int xrow = frow < M ? frow : M - 1;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int g = wave + kFusedWaves * t;
    if (g >= G) break;
    const v4i* px = reinterpret_cast<const v4i*>(codes + xrow * ld + g * 128 + 32 * fq);
    const int sx = *reinterpret_cast<const uint16_t*>(scales + (g * M + xrow) * 8 + 2 * fq);
    acc = mx_mfma<0>(w[t][0], px[0], acc, sw[t], sx);
    acc = mx_mfma<1>(w[t][1], px[1], acc, sw[t], sx);
  }
  v4f* part = reinterpret_cast<v4f*>(smem);         // the slots are free behind the barrier above
  part[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave) return;
  v4f y = part[lane];
#pragma unroll
  for (int v = 1; v < kFusedWaves; ++v) y += part[v * 64 + lane];
  const int64_t n = n0 + 4 * fq;
  if (frow >= M || n >= N) return;
  float bias[4], z[4] = {y[0], y[1], y[2], y[3]};
  load_bias(p, n, bias);
  finish<4>(p, z, frow, n, bias, n + 4 <= N);
}

// K = 0: every sum is empty.
__global__ void __launch_bounds__(256)
mx_empty_kernel(MxGemm p) {
  const int64_t total = p.M * p.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    float y = 0.0f;
    if (p.bias) y += p.bias[i % p.N];
    if (p.res) y += in16_to_f32(static_cast<const uint16_t*>(p.res)[i], p.bf16);
    static_cast<uint16_t*>(p.out)[i] =
        p.bf16 ? f32_to_bf16_rn(y) : __half_as_ushort(__float2half_rn(as_fp32(y)));
  }
}

// Row tiles per group of the tile order: 1024 rows, so that the workgroups
// resident on one XCD share a few bands of activations and panels of weights.
template <int WAM, int WAN, int FM, int FN, int ST>
hipError_t launch_tiles(const MxGemm& args, hipStream_t stream) {
  constexpr int BM = 32 * FM * WAM, BN = 32 * FN * WAN, NW = WAM * WAN;
  constexpr size_t lds = (size_t)ST * ((BM + BN) * 128 + ((BM + BN) / 32 + NW - 1) / NW * NW * 256);
  static_assert(lds <= 160 * 1024, "one CU's LDS");
  MxGemm a = args;
  a.group_m = 1024 / BM;
  const int64_t tiles = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  const auto fn = &mx_gemm_kernel<WAM, WAN, FM, FN, ST>;
  if (const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(fn), lds); e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((unsigned)tiles), dim3(64 * NW), lds, stream, a);
  return hipGetLastError();
}

template <int NB>
hipError_t launch_few(const MxGemm& a, hipStream_t stream) {
  hipLaunchKernelGGL((mx_few_kernel<NB, 8>), dim3((unsigned)((a.N + 15) / 16)), dim3(512), 0, stream, a);
  return hipGetLastError();
}

// Few rows, by size of the weights: the kernel without LDS tiles reads them in
// one round trip (1 row, 2048 x 2048: 3.4 us against 5.2; 4096 x 4096 4.4 against
// 7.1; 24 rows, 4096 x 8192 9.3 against 11.2), the tiles' direct loads stream
// large ones faster (4 rows, 16384 x 8192: 12.5 against 18; 24 rows, 8192 x 2048
// 5.4 against 6.1).
bool few_rows(int64_t M, int64_t N, int64_t K) {
  return M <= 16 ? N * K <= ((int64_t)1 << 26) : M <= 32 && N <= 4096;
}

}  // namespace

bool mx_fusable(int64_t M, int64_t N, int64_t K) {
  return K > 0 && M <= 16 && M * K <= kFusedGroups * kGroup && few_rows(M, N, K);
}

hipError_t launch_mx_fused(const MxGemm& a, const void* X, bool bf16, hipStream_t stream) {
  const auto fn = bf16 ? &mx_few_fused_kernel<true> : &mx_few_fused_kernel<false>;
  const size_t slots = (size_t)(a.M * (a.K / kGroup)) * kSlotBytes, sums = kFusedWaves * 64 * sizeof(v4f);
  const size_t lds = slots > sums ? slots : sums;
  if (const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(fn), lds); e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((unsigned)((a.N + 15) / 16)), dim3(64 * kFusedWaves), lds, stream, a,
                     static_cast<const uint16_t*>(X));
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemm& a, hipStream_t stream) {
  if (a.K == 0) {
    const int64_t blocks = (a.M * a.N + 255) / 256;
    hipLaunchKernelGGL(mx_empty_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (few_rows(a.M, a.N, a.K)) return a.M <= 16 ? launch_few<1>(a, stream) : launch_few<2>(a, stream);
  // Tiles: the largest that fill the card's 256 CUs (128x128 in 4 wavefronts and 70
  // KB runs twice on one), us: 8192^3 256x256 274, 128x128 315; 4096^3 47, 55;
  // 1024 x 8192 x 2048 128x128 15.8, 128x64 19.8; 1024 x 2048 x 8192 128x64 18.4 (no bias),
  // 64x64 20, 128x128 32; 777 x 1003 x 768 64x64 5.0, 128x64 6.0.
  const auto tiles = [&](int64_t bm, int64_t bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if (tiles(256, 256) >= 256) return launch_tiles<2, 4, 4, 2, 2>(a, stream);
  if (tiles(128, 128) >= 384) return launch_tiles<2, 2, 2, 2, 2>(a, stream);
  if (tiles(128, 64) >= 256) return launch_tiles<2, 2, 2, 1, 3>(a, stream);
  return launch_tiles<2, 2, 1, 1, 4>(a, stream);
}

}  // namespace convrot
