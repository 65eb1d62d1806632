// Host-side argument checks shared by the C entry points (internal to the library).
#pragma once

#include <atomic>
#include <cstring>

#include <hip/hip_runtime.h>

#include "convrot.h"

namespace convrot {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other / error
inline std::atomic<int> g_device_state[kMaxDevices];

inline convrot_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return CONVROT_ERR_DEVICE;
  int st = g_device_state[dev].load(std::memory_order_acquire);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      st = 2;
    } else {
      st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    }
    g_device_state[dev].store(st, std::memory_order_release);
  }
  return st == 1 ? CONVROT_OK : CONVROT_ERR_DEVICE;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// [a, a + na) and [b, b + nb) overlap?  (null or empty ranges never overlap)
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

inline convrot_status launched(hipError_t e) { return e == hipSuccess ? CONVROT_OK : CONVROT_ERR_LAUNCH; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace convrot
