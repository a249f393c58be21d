// txl_once.h -- host state of a kernel that belongs to a device: prepared once on each device of a process.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime_api.h>

namespace txl {

// Function attributes hold on the device that was current when they were set, so "once" means once per device.
// Threads may ask at the same time (both may then prepare: the same attributes twice); a failure is tried again.
class OncePerDevice {
public:
    template <typename F>
    cudaError_t operator()(F&& prepare)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return prepare();
        const uint64_t bit = uint64_t{1} << dev;
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = prepare();
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<uint64_t> done_{0};
};

// Lets the kernels take `bytes` of dynamic shared memory on the current device.
template <typename... K>
cudaError_t allow_smem(OncePerDevice& once, int bytes, K*... kernels)
{
    return once([&] {
        cudaError_t e = cudaSuccess;
        ((e = e == cudaSuccess ? cudaFuncSetAttribute(reinterpret_cast<const void*>(kernels),
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                               : e),
         ...);
        return e;
    });
}

}  // namespace txl
