// Argument checks that the C-ABI entry points of the operators around the dense
// head share.
#pragma once

#include <algorithm>
#include <cmath>
#include <exception>
#include <limits>

#include "fh_host.hpp"

namespace fh {

// No exception leaves a C entry (building an error text can throw).
template <typename R, typename F>
R guarded(R failed, F&& body) noexcept {
  try {
    g_err.clear();
    return body();
  } catch (const std::exception&) {
    return failed;
  }
}

inline bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int64_t kMaxElems = int64_t(1) << 60;    // rows * stride stays far inside int64

// The stride of `rows` rows of `width` elements, or an error text.
inline fh_status check_ld(const char* name, int64_t ld, int64_t width, int64_t rows) {
  if (ld < width)
    return fail(FH_EINVAL, std::string(name) + "=" + std::to_string(ld) + " below the row's " +
                               std::to_string(width) + " elements");
  if (ld > kMaxElems / rows) return fail(FH_EINVAL, std::string(name) + " too large");
  return FH_OK;
}

inline fh_status check_choice(int mode, float temperature) {
  if (mode != FH_TOKEN_ARGMAX && mode != FH_TOKEN_SAMPLE)
    return fail(FH_EINVAL, "mode must be FH_TOKEN_ARGMAX or FH_TOKEN_SAMPLE");
  if (mode == FH_TOKEN_SAMPLE && !(temperature > 0.f && std::isfinite(temperature)))
    return fail(FH_EINVAL, "sampling needs a finite temperature > 0");
  return FH_OK;
}

inline float inverse_of(float temperature) {
  return (float)std::min(1.0 / (double)temperature, (double)std::numeric_limits<float>::max());
}

inline fh_status check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  if (need == 0) return FH_OK;
  if (!workspace || bytes < need)
    return fail(FH_EINVAL, "this call needs " + std::to_string(need) + " bytes of workspace");
  if (!aligned16(workspace)) return fail(FH_EINVAL, "workspace must be 16-byte aligned");
  return FH_OK;
}

}  // namespace fh
