// Attention over the rotated, quantised key/value cache: which kernel runs a
// call, and its workspace.

#include "kv_core.hpp"

namespace convrot {
namespace {

// Rows (queries times heads of a group) per key head.  The few-row kernel
// decodes the cached rows anew for each 32 of them, in registers, and fills
// the card with few; the other shares the decoding among 128 or 256 through
// LDS.  Measured, few against many, us (heads of 128 in 4 bits, 8 key heads):
//   4 sequences of 8192 tokens:    40 rows 31 / 39, 72 rows 42 / 45, 128 rows 50 / 52, 192 rows 82 / 85
//   32 sequences of 2048 tokens:   40 rows 49 / 91, 72 rows 64 / 94, 128 rows 77 / 102, 256 rows 136 / 125
//   64 sequences of 512 tokens:    72 rows 53 / 55, 128 rows 60 / 58, 256 rows 111 / 72
bool few_rows(const KvAttn& a) { return (int64_t)a.max_q * a.group <= 128; }

}  // namespace

size_t kv_attention_workspace(const KvAttn& a) {
  return (few_rows(a) ? kv_decode_plan(a) : kv_prompt_plan(a)).bytes;
}

hipError_t launch_kv_attention(const KvAttn& a, void* workspace, hipStream_t stream) {
  return few_rows(a) ? launch_kv_decode(a, kv_decode_plan(a), workspace, stream)
                     : launch_kv_prompt(a, kv_prompt_plan(a), workspace, stream);
}

}  // namespace convrot
