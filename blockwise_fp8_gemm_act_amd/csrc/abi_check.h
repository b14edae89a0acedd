// Argument checks shared by the C ABI layers (host only): limits, alignment,
// overlaps, the device check, launch status.
#pragma once

#include "puro.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

namespace puro_abi {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxElems = int64_t(1) << 40;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  uintptr_t lo, hi;   // [lo, hi)
};

inline Range rng(const void *p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlap(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

// Any output overlapping any input or another output.
inline bool any_alias(const Range *in, int nin, const Range *out, int nout) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

inline bool shape_ok(int64_t r, int64_t c) {
  if (r < 0 || c < 0 || r > kMaxDim || c > kMaxDim) return false;
  if (r > 0 && c > kMaxElems / r) return false;
  return true;
}

// Per-device cache of the architecture check: 0 unknown, 1 gfx950, 2 other.
inline std::atomic<int> g_dev_ok[64];

inline puro_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return PURO_ERR_DEVICE;
  }
  if (dev < 64) {
    const int c = g_dev_ok[dev].load(std::memory_order_relaxed);
    if (c == 1) return PURO_OK;
    if (c == 2) return PURO_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    (void)hipGetLastError();
    return PURO_ERR_DEVICE;
  }
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < 64) g_dev_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? PURO_OK : PURO_ERR_DEVICE;
}

inline puro_status launched(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return PURO_ERR_LAUNCH;
  }
  return PURO_OK;
}

}  // namespace puro_abi
