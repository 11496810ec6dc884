// smem.cuh -- how much dynamic shared memory a kernel may be launched with.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace ssd {

// Per device, the bytes that a kernel has been allowed.  One object per kernel, static.
struct SmemLimit {
    std::atomic<int> bytes[64];
    std::mutex lock;
};

// Let a kernel take up to `bytes` of dynamic shared memory on the current device.  The limit only grows: calls of
// several threads ask for different sizes, and a smaller one that came between another's check and its launch, or
// between its setting and its record of it, would leave that launch refused.
template <typename F>
inline bool allow_smem(F *kernel, int bytes, SmemLimit &limit)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (limit.bytes[dev].load(std::memory_order_acquire) >= bytes) return true;
    const std::lock_guard<std::mutex> hold(limit.lock);
    if (limit.bytes[dev].load(std::memory_order_relaxed) >= bytes) return true;
    if (cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return false;
    limit.bytes[dev].store(bytes, std::memory_order_release);
    return true;
}

}  // namespace ssd
