// Launch helper of the block operators.
#pragma once

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace pdssm {

// Raises a kernel's dynamic shared-memory limit to `bytes` on the current
// device, once per device and size: `set` (one array per kernel, static)
// holds what each device was given.  Calls are short next to these launches.
// A limit is only ever raised, by one thread at a time: set and recorded out
// of step, a smaller limit could come to stand behind a larger one's launch.
constexpr int kLimitDevices = 64;
inline cudaError_t allow_smem(const void *kern, int bytes, std::atomic<int> (&set)[kLimitDevices]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kLimitDevices)
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (set[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    static std::mutex raising;
    const std::lock_guard<std::mutex> alone(raising);
    if (set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) set[dev].store(bytes, std::memory_order_release);
    return e;
}

}  // namespace pdssm
