// What is asked of the driver once for each device and kernel.
#pragma once

#include <atomic>

#include "dc_common.cuh"

namespace dc {

constexpr int kOnceDevices = 64;

// Allows `kern` its dynamic shared memory (always the same), the first time on
// each device; a further call costs a look at the current device.
template <typename K>
cudaError_t allow_smem_once(K kern, size_t bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev < kOnceDevices;
  if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace dc
