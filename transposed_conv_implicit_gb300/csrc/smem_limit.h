// Raises a kernel's dynamic shared-memory limit.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <mutex>

namespace convgb300 {

constexpr int kMaxDevices = 64;

// The limit is a function attribute, per device: raised to the largest size
// asked for so far, which `configured` (one entry per device and kernel)
// remembers.  Threads that raise it meet at a lock: a smaller size set after a
// larger one would leave the kernel a limit below what is remembered.
template <typename Kernel>
cudaError_t raise_smem(Kernel kernel, std::atomic<size_t>* configured, size_t smem) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (configured[dev].load(std::memory_order_acquire) >= smem) return cudaSuccess;
  static std::mutex raising;
  const std::lock_guard<std::mutex> lock(raising);
  if (configured[dev].load(std::memory_order_relaxed) >= smem) return cudaSuccess;
  err = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err == cudaSuccess) configured[dev].store(smem, std::memory_order_release);
  return err;
}

}  // namespace convgb300
