// Raises a kernel's dynamic shared-memory limit; how many of its blocks an SM runs.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
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

// Blocks of a kernel that an SM runs at once.  The last answer is remembered for each
// device and number of warps, with the shared memory that it was for: rows of other
// lengths may take more of it, and have their own answer.
constexpr int kWarpCounts = 33;
using BlocksPerSm = std::atomic<uint64_t>;  // shared memory << 16 | blocks
template <typename Kernel>
cudaError_t blocks_per_sm(Kernel kernel, BlocksPerSm (*known)[kWarpCounts], int threads, size_t smem, int* fit) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  BlocksPerSm& at = known[dev][threads / 32];
  const uint64_t last = at.load(std::memory_order_relaxed);
  *fit = static_cast<int>(last & 0xFFFFu);
  if (*fit > 0 && last >> 16 == smem) return cudaSuccess;
  err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(fit, reinterpret_cast<const void*>(kernel), threads, smem);
  if (err != cudaSuccess) return err;
  if (*fit < 1) *fit = 1;
  at.store(static_cast<uint64_t>(smem) << 16 | static_cast<uint64_t>(*fit), std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace convgb300
