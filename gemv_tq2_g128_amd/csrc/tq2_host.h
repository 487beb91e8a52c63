// Host-side argument checks shared by the C ABI translation units (not installed).
#pragma once

#include <atomic>
#include <cstring>

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tq2.h"

namespace tq2 {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other architecture.
inline std::atomic<int> g_device_kind[kMaxDevices];

inline int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return TQ2_ERR_DEVICE;
  if (dev < kMaxDevices) {
    const int kind = g_device_kind[dev].load(std::memory_order_relaxed);
    if (kind == 1) return TQ2_OK;
    if (kind == 2) return TQ2_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return TQ2_ERR_DEVICE;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDevices) g_device_kind[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? TQ2_OK : TQ2_ERR_DEVICE;
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? TQ2_OK : TQ2_ERR_LAUNCH; }

}  // namespace tq2
