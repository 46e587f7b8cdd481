// large_lds.hpp -- kernels that use more than 64 KiB of dynamic LDS: HIP is told
// so once per kernel and device (about a microsecond on the calling path each time).
// What is declared in a kernel does not count there.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace rt {

// `told`: one bit per device, one such word per kernel.
inline hipError_t allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &told) {
    int device = 0;
    hipError_t err = hipGetDevice(&device);
    if (err != hipSuccess) return err;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device < 64 && (told.load(std::memory_order_relaxed) & bit)) return hipSuccess;
    err = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == hipSuccess && device < 64) told.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

}  // namespace rt
