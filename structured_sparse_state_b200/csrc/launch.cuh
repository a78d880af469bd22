// Launch helper of the block operators.
#pragma once

#include <atomic>

#include "common.cuh"

namespace pdssm {

// Raises a kernel's dynamic shared-memory limit to `bytes` on the current
// device, once per device and size: `set` (one array per kernel, static)
// holds what each device was given.  Calls are short next to these launches.
constexpr int kLimitDevices = 64;
inline cudaError_t allow_smem(const void *kern, int bytes, std::atomic<int> (&set)[kLimitDevices]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kLimitDevices && set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < kLimitDevices) set[dev].store(bytes, std::memory_order_relaxed);
    return e;
}

}  // namespace pdssm
