// Host helpers shared by the C ABI's source files.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsai {

// IDX_EHIP, with the error's text kept for indexer_strerror (this thread).
int fail_hip(hipError_t e);

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    hipError_t err = hipSuccess;
    explicit DeviceGuard(int dev)
    {
        err = hipGetDevice(&prev);
        if (err == hipSuccess && prev != dev) {
            err = hipSetDevice(dev);
            changed = err == hipSuccess;
        }
    }
    ~DeviceGuard()
    {
        if (changed) (void)hipSetDevice(prev);
    }
};

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace dsai
