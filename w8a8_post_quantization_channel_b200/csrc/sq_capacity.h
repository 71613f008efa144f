// sq_capacity.h -- how many clusters of a kernel a device holds at once: asked
// once per device and kept.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace sq {

class CapacityCache {
 public:
  // *capacity on device `dev`, from ask(capacity) where it is not known yet.
  // A failed ask is this call's error and is not kept: the next call asks
  // again.  None fitting (0) is an answer like any other.  Threads that ask at
  // once keep the same value.
  template <class Ask>
  cudaError_t get(int dev, int *capacity, Ask ask) {
    std::atomic<int> *const kept = dev >= 0 && dev < kDevices ? &kept_[dev] : nullptr;
    if (kept != nullptr) {
      const int k = kept->load(std::memory_order_acquire);
      if (k != 0) {
        *capacity = k - 1;
        return cudaSuccess;
      }
    }
    int n = 0;
    const cudaError_t e = ask(&n);
    if (e != cudaSuccess) return e;
    *capacity = n > 0 ? n : 0;
    if (kept != nullptr) kept->store(*capacity + 1, std::memory_order_release);
    return cudaSuccess;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> kept_[kDevices] = {};  // capacity + 1; 0: not known
};

}  // namespace sq
