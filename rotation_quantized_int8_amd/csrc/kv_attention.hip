// Attention over the rotated, quantised key/value cache: which kernel runs a
// call, and its workspace.

#include "kv_core.hpp"

namespace convrot {

size_t kv_attention_workspace(const KvAttn& a) { return kv_decode_plan(a).bytes; }

hipError_t launch_kv_attention(const KvAttn& a, void* workspace, hipStream_t stream) {
  return launch_kv_decode(a, kv_decode_plan(a), workspace, stream);
}

}  // namespace convrot
