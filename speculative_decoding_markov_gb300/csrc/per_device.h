// per_device.h - what the library finds out or sets once per device: the limit
// of a kernel's dynamic shared memory, which cudaFuncSetAttribute raises on the
// current device alone, and the number of SMs.  Only successes are kept.
#pragma once
#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace sdm {

constexpr int kMaxDevices = 64;   // on those from here on the calls are made each time

// One kernel's limit, a static of the function that launches it.
class SmemLimit {
  public:
    // At least `bytes` on the current device; never lowered, whichever thread asks.
    template <typename... Args>
    cudaError_t raise(void (*kernel)(Args...), int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool known = dev >= 0 && dev < kMaxDevices;
        if (known && held_[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
        const std::lock_guard<std::mutex> lock(raising_);
        if (known && held_[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && known) held_[dev].store(bytes, std::memory_order_release);
        return e;
    }

  private:
    std::atomic<int> held_[kMaxDevices] = {};
    std::mutex raising_;
};

// SMs of the current device; 148 where there is none.
inline int sms_of_device() {
    static std::atomic<int> sms[kMaxDevices] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (known && (n = sms[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    if (known) sms[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace sdm
