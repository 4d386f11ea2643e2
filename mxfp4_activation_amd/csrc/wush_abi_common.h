// What the C-ABI files share: the error text of the last failure on this
// thread, pointer checks and the device check.
#ifndef WUSH_ABI_COMMON_H_
#define WUSH_ABI_COMMON_H_

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <atomic>

#include <hip/hip_runtime_api.h>

#include "../../include/wush.h"

namespace wush {

inline thread_local char g_last_error[512] = "";

inline wush_status fail(wush_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Half-open byte ranges [p, p + n) overlap?
inline bool overlap(const void* p, uint64_t np, const void* q, uint64_t nq) {
  if (!p || !q || np == 0 || nq == 0) return false;
  uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

// Per-device "is gfx950" cache: 0 unknown, 1 yes, 2 no.
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_dev_ok[kMaxDevices];

inline wush_status check_device() {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(WUSH_EHIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(WUSH_EUNSUPPORTED, "device index %d out of range", dev);
  int st = g_dev_ok[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return fail(WUSH_EHIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    st = (strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_dev_ok[dev].store(st, std::memory_order_relaxed);
  }
  if (st != 1) return fail(WUSH_EUNSUPPORTED, "device %d is not gfx950", dev);
  return WUSH_OK;
}

}  // namespace wush

#endif  // WUSH_ABI_COMMON_H_
