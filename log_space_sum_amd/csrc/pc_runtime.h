// pc_runtime.h -- error and device helpers shared by the C ABI's source files.
#pragma once
#include <hip/hip_runtime.h>

#include <string>

#include "pc_host.h"

namespace pc {

// Keeps the calling thread's message for pc_last_error and returns `code`.
int set_error(int code, const std::string& msg);

#define HIPCHECK(x)                                                                       \
  do {                                                                                    \
    hipError_t e_ = (x);                                                                  \
    if (e_ != hipSuccess) pc::fail(PC_ERR_HIP, std::string(#x) + ": " + hipGetErrorString(e_)); \
  } while (0)

// Makes `dev` the current device for its scope.
struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) prev = -1;
    if (prev != dev) HIPCHECK(hipSetDevice(dev));
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

inline void check_launch() {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) fail(PC_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

}  // namespace pc
