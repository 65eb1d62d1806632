// Host-side launchers of the norms around the linears (internal to the library).
#pragma once

#include "mx.hpp"

namespace convrot {

enum NormKind { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
enum NormOut { kOutNone = -1, kOut16 = 0, kOutInt8 = 1, kOutMx = 2 };

struct NormDesc {
  int kind;
  float eps;
  const float* weight;   // [D] or null
  const float* bias;     // [D] or null
};

struct NormArgs {
  const uint16_t* x;
  const uint16_t* y;              // the block's output (residual form) or null
  uint32_t x_stride, y_stride;    // elements, below 2^31 (32 bits: the kernel is short of scalar registers)
  uint32_t M;
  int D;
  float residual_scale;
  NormDesc post, norm;
  const void *scale, *shift, *gate;   // rows of the modulation or null
  uint32_t scale_stride, shift_stride, gate_stride;
  int mod_f32;                    // the modulation is fp32 (else the rows' type)
  uint32_t mod_rows;
  uint32_t each_mul;              // index null: row r has the modulation's row r each_mul >> each_shift,
  int each_shift;                 // r / each of each rows side by side (r < 2^31)
  float inv_d;                    // 1 / D
  double inv_wide;                // the same
  const int32_t* index;
  uint16_t* h;
  void* values;
  void* scales;
};

hipError_t launch_norm(const NormArgs& a, bool bf16, NormOut out, hipStream_t stream);
// The quantised forms (out kOutInt8 or kOutMx), by launch_norm.
hipError_t launch_norm_quant(const NormArgs& a, bool bf16, NormOut out, hipStream_t stream);

}  // namespace convrot
