// Host-side helpers shared by the translation units behind the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <exception>
#include <string>
#include <vector>

#include "muon.h"

namespace muon {

// Message of the last error on the calling thread (muon_last_error).
extern thread_local std::string g_last_error;

muon_status_t fail(muon_status_t st, const std::string& msg);
muon_status_t hip_fail(hipError_t e, const char* where);

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x, size_t a = kAlign) { return (x + a - 1) / a * a; }
inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool finite(float x) { return isfinite(x); }

// Byte range [lo, hi) of one buffer of a call; a writable one may overlap no
// other range of the call.
struct Range {
  uintptr_t lo, hi;
  bool writable;
  const char* what;
  int64_t idx;
};
muon_status_t check_aliasing(std::vector<Range>& rs);

// Runs the body of a C entry point, turning an exception (host memory ran out) into an error.
template <class F>
muon_status_t guarded(F&& f) noexcept {
  g_last_error.clear();
  try {
    return f();
  } catch (const std::exception&) {
    return MUON_ERR_HIP;  // the message, too, would need memory
  }
}

}  // namespace muon
