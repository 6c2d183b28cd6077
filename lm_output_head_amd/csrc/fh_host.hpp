// Host-side helpers of the C-ABI entry points: the thread's error text, and a
// guard that selects a device for one call.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "flashhead.h"

namespace fh {

extern thread_local std::string g_err;

// Set the thread's error text; return st.
fh_status fail(fh_status st, const std::string& msg);
// The same for a failed HIP call, whose error the runtime also keeps until it is
// read: that one is consumed.  FH_ENOMEM or FH_EHIP.
fh_status hip_fail(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    ok = hipGetDevice(&prev) == hipSuccess && (prev == dev || hipSetDevice(dev) == hipSuccess);
    if (!ok) (void)hipGetLastError();  // the call reports it
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

}  // namespace fh
