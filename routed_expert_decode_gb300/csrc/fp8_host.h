// fp8_host.h -- host-side state that the fp8 launchers keep per device.  Calls from
// several host threads may overlap: every thread that finds an entry unset gives the
// driver and the entry the same value.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>

namespace moe {

constexpr int kMaxDevices = 64;
constexpr size_t kSmemLimit = 232448;  // shared memory of a CTA

// the current device, -1 when there is none (or it is past kMaxDevices)
inline int device_here() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices ? dev : -1;
}

// Let `kern`, which has no static shared memory, take all that a CTA has as dynamic
// shared memory on the current device: the same for every call, so that calls of
// different sizes cannot undo each other's.  `done`: kMaxDevices of the kernel's own.
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<bool> *done) {
  const int dev = device_here();
  if (dev >= 0 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      (const void *)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
  if (e == cudaSuccess && dev >= 0) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

}  // namespace moe
