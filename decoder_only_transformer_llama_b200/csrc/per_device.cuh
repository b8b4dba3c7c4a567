// Host state that a launcher keeps for each device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace llb {

// What a launcher asks of the device or sets on it once: a kernel's attributes
// hold on the device they were set on.  Any host thread may be the first.
template <typename V>
class PerDevice {
  public:
    // *out = the current device's value, filled by make(device, out) on the first call there.
    template <typename F>
    cudaError_t get(V* out, F make) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kDevices) return make(dev, out);
        if (!ready_[dev].load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> lock(mu_);
            if (!ready_[dev].load(std::memory_order_relaxed)) {
                e = make(dev, &value_[dev]);
                if (e != cudaSuccess) return e;
                ready_[dev].store(true, std::memory_order_release);
            }
        }
        *out = value_[dev];
        return cudaSuccess;
    }

  private:
    static constexpr int kDevices = 64;
    std::mutex mu_;
    std::atomic<bool> ready_[kDevices] = {};
    V value_[kDevices] = {};
};

}  // namespace llb
