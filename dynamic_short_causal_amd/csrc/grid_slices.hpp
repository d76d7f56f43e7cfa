// grid_slices.hpp -- calls of more threads than one launch can have.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsc {

// A launch counts its threads in 32 bits and drops what is above, without an error.
constexpr int64_t kLaunchThreads = UINT32_MAX;

// For kernels that take their workgroups in one launch: others are refused.
inline hipError_t one_launch(int64_t groups, int threads) {
  return groups <= kLaunchThreads / threads ? hipSuccess : hipErrorInvalidConfiguration;
}

// Calls launch(first, n) for workgroups first .. first + n - 1 of `groups`, with
// fewer than 2^32 threads each time: once, but for the largest calls.
template <typename F> hipError_t launch_slices(int64_t groups, int threads, F launch) {
  const int64_t most = kLaunchThreads / threads;
  for (int64_t first = 0; first < groups; first += most) {
    launch((uint32_t)first, dim3((unsigned)(groups - first < most ? groups - first : most)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace dsc
