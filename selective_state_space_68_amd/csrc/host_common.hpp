// Helpers of the C-ABI host layer: address ranges and their overlap, overflow-checked
// sizes, the cached device probe.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/ssm.h"

namespace ssm {

struct Span {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
  bool empty() const { return lo == hi; }
};

inline Span span(const void* p, uint64_t bytes) {
  Span s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + (p ? bytes : 0);
  return s;
}

inline bool overlaps(const Span& a, const Span& b) {
  if (a.empty() || b.empty()) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline bool mul_ok(uint64_t a, uint64_t b, uint64_t* out) { return !__builtin_mul_overflow(a, b, out); }

inline bool aligned(const void* p, uintptr_t a) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 1 = a device is usable, 0 = none; probed once per process.
inline std::atomic<int> g_device_state{-1};

inline ssm_status probe_device() {
  int st = g_device_state.load(std::memory_order_relaxed);
  if (st == 1) return SSM_OK;
  if (st == 0) return SSM_ERR_HIP;
  int count = 0;
  const hipError_t e = hipGetDeviceCount(&count);
  st = (e == hipSuccess && count > 0) ? 1 : 0;
  if (e != hipSuccess) (void)hipGetLastError();
  g_device_state.store(st, std::memory_order_relaxed);
  return st ? SSM_OK : SSM_ERR_HIP;
}

inline ssm_status from_hip(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

}  // namespace ssm
