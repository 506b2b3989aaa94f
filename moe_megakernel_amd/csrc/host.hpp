// Host-side helpers shared by the units that implement C entry points: alignment checks,
// the per-kernel timer and the launch wrapper.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/moe.h"

namespace moe {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// at a multiple of its elements' size (MOE_BF16 or MOE_FP32)
inline bool elem_aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_BF16 ? 1u : 3u)) == 0;
}

// ---------------------------------------------------------------- kernel timer
struct TimedLaunch {
  const char* name;
  hipEvent_t a, b;
};
struct Timer {
  bool on = false;
  std::vector<TimedLaunch> pending;
  std::vector<hipEvent_t> pool;
  std::vector<std::string> names;
  std::vector<int> counts;
  std::vector<double> ms;
  std::mutex mu;
  hipEvent_t get() {
    if (!pool.empty()) { hipEvent_t e = pool.back(); pool.pop_back(); return e; }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
  }
};
inline Timer g_timer;

template <class F>
moe_status launch(const char* name, hipStream_t st, F&& f) {
  hipEvent_t a = nullptr, b = nullptr;
  if (g_timer.on) {
    a = g_timer.get();
    b = g_timer.get();
    if (a) (void)hipEventRecord(a, st);
  }
  f();
  const hipError_t err = hipGetLastError();
  if (g_timer.on && a && b) {
    (void)hipEventRecord(b, st);
    g_timer.pending.push_back({name, a, b});
  }
  return err == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

#define MOE_TRY(x)                        \
  do {                                    \
    const moe_status _s = (x);            \
    if (_s != MOE_OK) return _s;          \
  } while (0)

}  // namespace moe
