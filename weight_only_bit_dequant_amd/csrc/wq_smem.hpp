// Leave for dynamic LDS above 64 KiB, asked for once per kernel and device.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <atomic>

namespace wq {

// Devices on which a kernel has its leave, a bit each.
using SmemAllowed = std::atomic<uint64_t>;

// The attribute belongs to the kernel as the current device has it: a process
// that drives several GPUs asks on each.
template <typename Kern>
hipError_t allow_smem(Kern k, int bytes, SmemAllowed& done) {
  if (bytes <= 65536) return hipSuccess;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;  // (past 64 devices: asked for at every launch)
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace wq
