// Attention over the rotated, quantised key/value cache: which kernel runs a
// call, and its workspace.

#include "kv_core.hpp"

namespace convrot {
namespace {

// Up to 32 rows (queries times heads of a group) per key head the cached rows
// are read for one or two tiles of 16: HBM counts, and the single-token
// kernel decodes in registers.  More rows share the decoding through LDS.
bool few_rows(const KvAttn& a) { return (int64_t)a.max_q * a.group <= 32; }

}  // namespace

size_t kv_attention_workspace(const KvAttn& a) {
  return (few_rows(a) ? kv_decode_plan(a) : kv_prompt_plan(a)).bytes;
}

hipError_t launch_kv_attention(const KvAttn& a, void* workspace, hipStream_t stream) {
  return few_rows(a) ? launch_kv_decode(a, kv_decode_plan(a), workspace, stream)
                     : launch_kv_prompt(a, kv_prompt_plan(a), workspace, stream);
}

}  // namespace convrot
