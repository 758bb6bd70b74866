// Checks shared by the C-ABI entry points: device gate, alignment, overlap.
#pragma once

#include <stdint.h>

#include <atomic>

#include "internal.h"

namespace h3 {

constexpr int kMaxDevices = 64;

// Per device: 0 = not yet known, 1 = supported, 2 = not supported.  Stored
// only after both attribute queries succeeded, so a failed query is retried
// on the next call instead of marking the device unsupported for good.
inline std::atomic<int> g_dev_state[kMaxDevices];

// Gate on compute capability 10.3 (the only target the kernels are built for).
inline h3attn_status_t check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return H3ATTN_ERR_LAUNCH;
  if (dev < 0 || dev >= kMaxDevices) return H3ATTN_ERR_UNSUPPORTED_DEVICE;
  int state = g_dev_state[dev].load(std::memory_order_acquire);
  if (state == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return H3ATTN_ERR_LAUNCH;
    state = (major == 10 && minor == 3) ? 1 : 2;
    g_dev_state[dev].store(state, std::memory_order_release);  // racing callers store the same value
  }
  return state == 1 ? H3ATTN_OK : H3ATTN_ERR_UNSUPPORTED_DEVICE;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(nb) && b0 < a0 + static_cast<uintptr_t>(na);
}

inline bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

}  // namespace h3
