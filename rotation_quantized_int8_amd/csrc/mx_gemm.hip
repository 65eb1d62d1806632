// The product of microscaled 4-bit rows, Y = out(X W^T + bias + residual), on
// the scaled matrix instructions of gfx950.
//
// Mathematics.  v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows
// over 128 elements, four blocks of 32 with a scale each: a lane holds one
// block of one row (16 bytes) and, in a byte of a register, its scale.  The sum
// over K does not ask which block a lane takes, as long as both operands agree:
// of a rotation group (8 blocks, 128 bytes a row) lane quarter q takes blocks 2q
// and 2q + 1, one an instruction, so that its two scales are neighbouring bytes
// of the layout [K / 256, rows, 8] and one 16-bit read serves both instructions.
//
// Data flow.  Tiles as in the int8 product: direct global->LDS loads into a ring
// of STAGES slices of one rotation group, 16-byte chunks XOR-swizzled by row & 7
// (conflict-free fills and reads); the slice's scales, 8 bytes a row, follow the
// codes in the same ring.  The weight tile is the left operand, so a lane's four
// accumulators are four neighbouring outputs of one row.
//
// Rows past M or N repeat the last valid row for the loads and are dropped in
// the epilogue.

#include "dma.hpp"
#include "mx.hpp"

namespace convrot {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

// acc += (w 2^sw) (x 2^sx)^T; byte kk of the registers sw and sx.
template <int kk>
__device__ __forceinline__ v4f mx_mfma(v4i w, v4i x, v4f acc, int sw, int sx) {
  const v8i a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, kk, sw, kk, sx);   // 4: e2m1
}

__device__ __forceinline__ float in16_to_f32(uint16_t bits, int bf16) {
  return bf16 ? bf16_to_f32(bits) : __half2float(__ushort_as_half(bits));
}

// Four neighbouring outputs (row m, columns n ..) from finished sums: bias and
// residual added in fp32, one rounding; columns past N give anything.
__device__ __forceinline__ uint2 mx_finish(const MxGemm& p, v4f y, int64_t m, int64_t n, const float (&bias)[4]) {
  if (p.bias) {
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] += bias[r];
  }
  if (p.res) {
    const uint16_t* src = static_cast<const uint16_t*>(p.res) + m * p.N + n;
    uint16_t h[4];
    if ((p.N & 3) == 0 && n < p.N) {
      const uint2 t = *reinterpret_cast<const uint2*>(src);
      h[0] = t.x & 0xFFFF;
      h[1] = t.x >> 16;
      h[2] = t.y & 0xFFFF;
      h[3] = t.y >> 16;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = n + r < p.N ? src[r] : 0;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] += in16_to_f32(h[r], p.bf16);
  }
  uint2 v;
  if (p.bf16) {
    v.x = (uint32_t)f32_to_bf16_rn(y[0]) | (uint32_t)f32_to_bf16_rn(y[1]) << 16;
    v.y = (uint32_t)f32_to_bf16_rn(y[2]) | (uint32_t)f32_to_bf16_rn(y[3]) << 16;
  } else {
    v.x = pack_f16x2_rn(y[0], y[1]);
    v.y = pack_f16x2_rn(y[2], y[3]);
  }
  return v;
}

template <int WAVES_M, int WAVES_N, int FM, int FN, int STAGES>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N)
mx_gemm_kernel(MxGemm p) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = 16 * FM, WN = 16 * FN;
  constexpr int BM = WAVES_M * WM, BN = WAVES_N * WN;
  constexpr int XL = BM / 8 / NW, WL = BN / 8 / NW;               // 1 KiB blocks (8 rows) a wave loads per slice
  constexpr int SL = ((BM + BN) / 32 + NW - 1) / NW;              // 256-byte blocks of scales (32 rows)
  constexpr int LPW = XL + WL + SL;
  constexpr int XBYTES = BM * 128, WBYTES = BN * 128, SBYTES = SL * NW * 256;
  constexpr int STAGE = XBYTES + WBYTES + SBYTES;
  constexpr int kAhead = (STAGES - 2) * LPW;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && (BM + BN) % 32 == 0, "blocks split evenly over waves");
  static_assert(STAGES >= 2 && kAhead < 64, "pipeline depth");

  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int64_t M = p.M, N = p.N, nk = p.K / kGroup, ld = p.K / 2;
  const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN, T = tiles_m * tiles_n;
  int64_t t;
  {
    const int64_t b = blockIdx.x, x = b & 7, i = b >> 3, per = T >> 3, rem = T & 7;
    t = x * per + (x < rem ? x : rem) + i;
  }
  const int64_t in_group = p.group_m * tiles_n;
  const int64_t first_m = (t / in_group) * p.group_m;
  const int64_t gsize = (tiles_m - first_m) < p.group_m ? (tiles_m - first_m) : p.group_m;
  const int64_t m0 = (first_m + (t % in_group) % gsize) * BM, n0 = ((t % in_group) / gsize) * BN;

  const char* srcx[XL];
  const char* srcw[WL];
  const char* srcs[SL];
  int64_t steps[SL];   // bytes from one group's scales to the next group's
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = 8 * (wave * XL + i) + (lane >> 3);
    const int64_t row = m0 + r < M ? m0 + r : M - 1;
    srcx[i] = reinterpret_cast<const char*>(p.x) + row * ld + 16 * ((lane & 7) ^ (r & 7));
  }
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int r = 8 * (wave * WL + i) + (lane >> 3);
    const int64_t row = n0 + r < N ? n0 + r : N - 1;
    srcw[i] = reinterpret_cast<const char*>(p.w) + row * ld + 16 * ((lane & 7) ^ (r & 7));
  }
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int r = 32 * (wave * SL + i) + (lane >> 1);
    const bool of_x = r < BM;      // rows past both tiles repeat the last weight row
    const int64_t first = of_x ? m0 + r : n0 + r - BM, rows = of_x ? M : N;
    const int64_t row = first < rows ? first : rows - 1;
    srcs[i] = reinterpret_cast<const char*>(of_x ? p.xs : p.ws) + row * 8 + 4 * (lane & 1);
    steps[i] = rows * 8;
  }
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
  auto issue = [&](int64_t kt) {
    const uint32_t at = lds_base + ((uint32_t)kt % STAGES) * STAGE;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      dma16(srcx[i] + kt * 128, __builtin_amdgcn_readfirstlane(at + (wave * XL + i) * 1024));
#pragma unroll
    for (int i = 0; i < WL; ++i)
      dma16(srcw[i] + kt * 128, __builtin_amdgcn_readfirstlane(at + XBYTES + (wave * WL + i) * 1024));
#pragma unroll
    for (int i = 0; i < SL; ++i)
      dma4(srcs[i] + kt * steps[i],
           __builtin_amdgcn_readfirstlane(at + XBYTES + WBYTES + (wave * SL + i) * 256));
  };

  v4f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  const int frow = lane & 15, fq = lane >> 4;
  v4i fw[FN], fx[FM];
  int sw[FN], sx[FM];
  auto load_scales = [&](const char* st) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
      sw[i] = *reinterpret_cast<const uint16_t*>(st + XBYTES + WBYTES + (BM + wn * WN + i * 16 + frow) * 8 + 2 * fq);
#pragma unroll
    for (int j = 0; j < FM; ++j)
      sx[j] = *reinterpret_cast<const uint16_t*>(st + XBYTES + WBYTES + (wm * WM + j * 16 + frow) * 8 + 2 * fq);
  };
  auto load_frags = [&](const char* st, int kk) {
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int row = wn * WN + i * 16 + frow;
      fw[i] = *reinterpret_cast<const v4i*>(st + XBYTES + row * 128 + 16 * ((2 * fq + kk) ^ (row & 7)));
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int row = wm * WM + j * 16 + frow;
      fx[j] = *reinterpret_cast<const v4i*>(st + row * 128 + 16 * ((2 * fq + kk) ^ (row & 7)));
    }
  };

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < nk) issue(s);
  for (int64_t kt = 0; kt < nk; ++kt) {
    // slice kt has landed for this wave once only the later ones are in flight;
    // the barrier publishes every wave's part and frees the slice before it
    if (kt + STAGES - 2 < nk) wait_vmcnt<kAhead>();
    else wait_vmcnt<0>();
    lds_barrier();
    if (kt + STAGES - 1 < nk) issue(kt + STAGES - 1);
    const char* st = smem + ((uint32_t)kt % STAGES) * STAGE;
    load_scales(st);
    load_frags(st, 0);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = mx_mfma<0>(fw[i], fx[j], acc[i][j], sw[i], sx[j]);
    load_frags(st, 1);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = mx_mfma<1>(fw[i], fx[j], acc[i][j], sw[i], sx[j]);
  }

  // The finished tile goes through LDS (the ring is free behind the barrier), so
  // that stores are whole 16-byte chunks of output rows.  A residual is read
  // here, by the workgroup that writes its tile, before the barrier: it may be
  // the output.
  constexpr int ROWB = BN * 2 + 16;
  static_assert(BM * ROWB <= STAGES * STAGE, "the staged tile must fit in the ring");
  lds_barrier();
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int nl = wn * WN + i * 16 + 4 * fq;
    float bias[4] = {0, 0, 0, 0};
    if (p.bias) {
#pragma unroll
      for (int r = 0; r < 4; ++r) bias[r] = p.bias[n0 + nl + r < N ? n0 + nl + r : N - 1];
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int ml = wm * WM + j * 16 + frow;
      const int64_t m = m0 + ml < M ? m0 + ml : M - 1;
      *reinterpret_cast<uint2*>(smem + ml * ROWB + nl * 2) = mx_finish(p, acc[i][j], m, n0 + nl, bias);
    }
  }
  lds_barrier();
  constexpr int CPR = BN / 8;   // 16-byte chunks of a tile row
  uint16_t* out = static_cast<uint16_t*>(p.out);
  for (int c = tid; c < BM * CPR; c += 64 * NW) {
    const int rl = c / CPR, cc = c - rl * CPR;
    const int64_t m = m0 + rl, n = n0 + cc * 8;
    if (m >= M || n >= N) continue;
    const char* sp = smem + rl * ROWB + cc * 16;
    uint16_t* gp = out + m * N + n;
    if ((N & 7) == 0) {
      __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(sp), reinterpret_cast<v4i*>(gp));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) gp[e] = reinterpret_cast<const uint16_t*>(sp)[e];
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
  float bias[4] = {0, 0, 0, 0};
  if (p.bias) {
#pragma unroll
    for (int r = 0; r < 4; ++r) bias[r] = p.bias[n + r < N ? n + r : N - 1];
  }
  const uint2 v = mx_finish(p, y, m, n, bias);
  uint16_t* out = static_cast<uint16_t*>(p.out) + m * N + n;
  if ((N & 3) == 0) {
    *reinterpret_cast<uint2*>(out) = v;
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) out[r] = (uint16_t)((r < 2 ? v.x : v.y) >> (16 * (r & 1)));
  }
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
  constexpr int BM = 16 * FM * WAM, BN = 16 * FN * WAN, NW = WAM * WAN;
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

}  // namespace

hipError_t launch_mx_gemm(const MxGemm& a, hipStream_t stream) {
  if (a.K == 0) {
    const int64_t blocks = (a.M * a.N + 255) / 256;
    hipLaunchKernelGGL(mx_empty_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (a.M <= 16) return launch_few<1>(a, stream);
  if (a.M <= 32) return launch_few<2>(a, stream);
  const auto tiles = [&](int64_t bm, int64_t bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if (tiles(256, 256) >= 256) return launch_tiles<2, 4, 8, 4, 2>(a, stream);
  if (tiles(128, 128) >= 256) return launch_tiles<2, 2, 4, 4, 2>(a, stream);
  return launch_tiles<2, 2, 2, 2, 4>(a, stream);
}

}  // namespace convrot
