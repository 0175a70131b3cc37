// tfp8_host.hpp - what the C entry points share on the host: argument checks, the device's count of
// compute units, and the launch itself.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <tuple>

#include "../../include/tfp8.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void *p, int64_t bytes) {
  return Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool target_ok(float t) {
  return isfinite(t) && t >= 0x1p-64f && t <= 0x1p64f;
}

inline int cu_count() {
  // compute units of the current device, looked up once per device (any thread may race to
  // fill an entry; they all store the same value)
  constexpr int kMaxDevices = 64;
  static std::atomic<int> by_device[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  int cus = by_device[dev].load(std::memory_order_relaxed);
  if (cus <= 0) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
        cus <= 0)
      cus = 256;
    by_device[dev].store(cus, std::memory_order_relaxed);
  }
  return cus;
}

// Launches `kernel` with `args` converted to its parameter types, and returns the status of this
// launch itself (hipLaunchKernel reports it directly, so an error left over from an earlier,
// unrelated HIP call is not taken for this launch's).
template <typename... KArgs, typename... Args>
tfp8_status launch(void (*kernel)(KArgs...), unsigned grid, int threads, hipStream_t st,
                   Args... args) {
  static_assert(sizeof...(KArgs) == sizeof...(Args), "kernel argument count");
  std::tuple<KArgs...> held(static_cast<KArgs>(args)...);
  void *argv[sizeof...(KArgs)];
  std::apply([&argv](auto &...a) {
    int i = 0;
    ((argv[i++] = (void *)&a), ...);
  }, held);
  return hipLaunchKernel((const void *)kernel, dim3(grid), dim3(threads), argv, 0, st) ==
                 hipSuccess
             ? TFP8_OK
             : TFP8_E_HIP;
}

}  // namespace
