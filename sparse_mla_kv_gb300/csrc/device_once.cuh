// What a process does once for each device, such as raising a kernel's shared-memory limit (the attribute belongs to the
// device, not to the process).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace hs {

class DeviceOnce {
 public:
  // Runs prepare() unless it has succeeded for this device before.  A failure is returned and not kept: the next call tries
  // again.  Threads that come first together may all run it.
  template <typename F>
  cudaError_t ready(int dev, F prepare) {
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = prepare();
    if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> done_[kDevices] = {};
};

}  // namespace hs
