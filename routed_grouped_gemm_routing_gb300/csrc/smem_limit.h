// Raises a kernel's limit of dynamic shared memory, once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "moe_internal.h"

namespace moe {

// One static object per kernel: more than 48 KB of dynamic shared memory has
// to be asked for before the first launch on each device.  Host threads may
// race to ask for the same value.
struct SmemLimit {
    std::atomic<bool> done[kMaxDevices] = {};
    template <typename K>
    int allow(K kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return (int)e;
        if (dev < 0 || dev >= kMaxDevices) return (int)cudaErrorInvalidDevice;
        if (done[dev].load(std::memory_order_relaxed)) return 0;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
        return (int)e;
    }
};

}  // namespace moe
