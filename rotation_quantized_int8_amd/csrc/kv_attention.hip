// Attention over the rotated, quantised key/value cache: which kernel runs a
// call, and its workspace.

#include "kv_core.hpp"

namespace convrot {
namespace {

// Rows (queries times heads of a group) per key head.  The few-row kernel
// decodes the cached rows anew for each 32 of them, in registers, and fills
// the card with few; the other shares the decoding among 128 or 256 through
// LDS.  Measured, few against many, us (heads of 128 in 4 bits, 8 key heads):
//   4 sequences of 8192 tokens:    40 rows 31 / 39, 72 rows 42 / 44, 128 rows 51 / 51, 192 rows 82 / 85
//   32 sequences of 2048 tokens:   40 rows 41 / 81, 72 rows 60 / 78, 128 rows 72 / 80, 256 rows 136 / 125
//   64 sequences of 512 tokens:    40 rows 33 / 52, 72 rows 46 / 54, 128 rows 60 / 58, 256 rows 111 / 72
//   1 sequence of 300 tokens:      40 rows 12 / 17, 128 rows 12 / 19
//   4 of 8192, heads of 256:       40 rows 49 / 101, 128 rows 82 / 138, 256 rows 243 / 209
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
