// Host-side checks shared by the C ABI files (api.cpp, api_moe.cpp).
#pragma once

#include "../../include/fp8blk.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

namespace fp8blk {

constexpr int64_t kGroup = 128;
constexpr int kMaxDevices = 64;
// Once-initialised per-device answer to "is this a gfx950?": 0 unknown, 1 yes, 2 no.
inline std::atomic<int> g_device_ok[kMaxDevices];

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool mult128(int64_t v) { return v > 0 && v % kGroup == 0; }
// a * b <= limit for a, b > 0, without forming the (possibly overflowing) product
inline bool prod_le(int64_t a, int64_t b, int64_t limit) { return a <= limit / b; }
// a * b < limit, likewise
inline bool prod_lt(int64_t a, int64_t b, int64_t limit) { return a < (limit + b - 1) / b; }
inline bool valid_scale_mode(int m) { return m == FP8BLK_SCALE_POW2 || m == FP8BLK_SCALE_FP32; }

inline int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return FP8BLK_ERR_HIP;
  if (dev < 0 || dev >= kMaxDevices) return FP8BLK_ERR_DEVICE;
  int known = g_device_ok[dev].load(std::memory_order_acquire);
  if (known == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8BLK_ERR_HIP;
    known = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_device_ok[dev].store(known, std::memory_order_release);
  }
  return known == 1 ? FP8BLK_OK : FP8BLK_ERR_DEVICE;
}

inline int finish(hipError_t e) { return e == hipSuccess ? FP8BLK_OK : FP8BLK_ERR_HIP; }

// Largest element count the 32-bit index arithmetic inside the kernels covers.
constexpr int64_t kMaxElems = int64_t(1) << 40;

}  // namespace fp8blk
