// A kernel's limit of dynamic shared memory, raised once per device.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fa {

// One per kernel (a static of the function that launches it).  Devices past
// the 64th are raised on every call.
struct SmemLimit {
  std::atomic<uint64_t> raised{0};
  template <typename Kernel>
  cudaError_t raise(Kernel kern, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (raised.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) raised.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

}  // namespace fa
