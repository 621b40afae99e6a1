// A step that a device needs once (a kernel's dynamic shared-memory limit belongs to the
// current device), taken again where it failed: an error is the failing call's own.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>

namespace relation {

class OncePerDevice {
  public:
    template <typename Step>
    cudaError_t run(int device, Step step) {
        if (device < 0 || device >= kDevices) return cudaErrorInvalidDevice;
        if (done_[device].load(std::memory_order_acquire)) return cudaSuccess;
        std::lock_guard<std::mutex> lock(mutex_);
        if (done_[device].load(std::memory_order_relaxed)) return cudaSuccess;
        const cudaError_t e = step();
        if (e == cudaSuccess) done_[device].store(true, std::memory_order_release);
        return e;
    }

  private:
    static constexpr int kDevices = 64;
    std::mutex mutex_;
    std::atomic<bool> done_[kDevices] = {};
};

// Lets kern ask for `bytes` of dynamic shared memory on the current device; once: the kernel's own.
template <typename Kernel>
cudaError_t allow_dynamic_smem(OncePerDevice& once, Kernel* kern, int bytes) {
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return once.run(device,
                    [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}

// Splits an SM between shared memory and L1 so that `blocks` of kern's blocks, of `bytes` each, fit on the current
// device, and no further; once: the kernel's own. Left alone, an SM keeps the split of the kernel before.
template <typename Kernel>
cudaError_t prefer_shared(OncePerDevice& once, Kernel* kern, int blocks, int bytes) {
    int device = 0, most = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return once.run(device, [&] {
        if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerMultiprocessor, device)) != cudaSuccess) return e;
        const int percent = std::min(100, (100 * blocks * (bytes + 1024) + most - 1) / most);  // (1 KB is the system's)
        return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, percent);
    });
}

}  // namespace relation
