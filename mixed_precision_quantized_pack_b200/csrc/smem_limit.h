// A kernel's limit of dynamic shared memory.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>

namespace kvq {

// Raises a kernel's limit on the current device to the largest size asked for so far, once (a call to
// the runtime each time costs more than the launch's argument checks).  Caches on several host
// threads launch the same kernels with different sizes, so the attribute is set and recorded under one
// lock and never lowered: a smaller size set behind the record of a larger one would fail every
// later launch of the larger.
struct SmemLimit {
  static constexpr int kDevices = 64;         // devices past these set the attribute in every call
  std::atomic<int> bytes[kDevices] = {};
  std::mutex lock;
  int most = 0;

  cudaError_t raise(const void* kernel, int need) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (known && bytes[dev].load(std::memory_order_acquire) >= need) return cudaSuccess;
    const std::lock_guard<std::mutex> hold(lock);
    if (known && bytes[dev].load(std::memory_order_relaxed) >= need) return cudaSuccess;
    const int size = std::max(most, need);
    const cudaError_t e2 = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, size);
    if (e2 != cudaSuccess) return e2;
    most = size;
    if (known) bytes[dev].store(size, std::memory_order_release);
    return cudaSuccess;
  }
  template <typename... Args>
  cudaError_t raise(void (*kernel)(Args...), int need) {
    return raise(reinterpret_cast<const void*>(kernel), need);
  }
};

}  // namespace kvq
