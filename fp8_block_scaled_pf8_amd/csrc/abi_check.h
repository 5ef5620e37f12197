// What the C ABI's layers share on the host: argument checks and statuses.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pf8.h"

namespace pf8 {

// Every dimension, pitch and stride is at most 2^31 - 1 (PF8_ESHAPE otherwise), so that sizes in bytes stay
// far below 2^63.
constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
template <typename... T>
bool any_too_big(T... v) {
  return ((v > kMaxDim) || ...);
}

// A GEMM tile's rows are addressed from its first by signed 32-bit offsets: 256 rows x pitch in bytes.
constexpr int64_t kMaxTilePitch = kMaxDim / 256;

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline int device_status() {
  int count = 0;
  if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) {
    (void)hipGetLastError();  // clear the sticky error of a failed query
    return PF8_ENODEV;
  }
  return PF8_OK;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? PF8_OK : PF8_ELAUNCH; }

}  // namespace pf8
