// lores_host.h -- host helpers shared by the library's C entry points.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "lores.h"

namespace {

struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev == dev) {                 // the usual case: nothing to set, nothing to restore
      prev = -1;
      ok = true;
    } else {
      ok = cudaSetDevice(dev) == cudaSuccess;
    }
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline lores_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return LORES_OK;
  if (e == cudaErrorMemoryAllocation) {
    (void)cudaGetLastError();
    return LORES_ERR_OOM;
  }
  return LORES_ERR_CUDA;
}

}  // namespace
