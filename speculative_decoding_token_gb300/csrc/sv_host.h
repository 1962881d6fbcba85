// sv_host.h -- what the host sides of the C ABI share (not part of it): the device
// of a call, and what a CUDA error becomes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "specverify.h"

namespace sv {

constexpr uint64_t kDefaultWaitNs = 2000000000ull;  // bound of a wait inside a kernel: about two seconds

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    cudaError_t err = cudaSuccess;
    explicit DeviceGuard(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            changed = err == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

inline int map_cuda(cudaError_t e) {
    if (e == cudaSuccess) return SPECVERIFY_OK;
    cudaGetLastError();  // it is reported here: the program's next launch check need not see it
    if (e == cudaErrorMemoryAllocation) return SPECVERIFY_ERR_OOM;
    return SPECVERIFY_ERR_CUDA;
}

// Whether the machine has that device.
inline int check_device(int device) {
    int ndev = 0;
    const int rc = map_cuda(cudaGetDeviceCount(&ndev));
    return rc == SPECVERIFY_OK && device >= ndev ? SPECVERIFY_ERR_CUDA : rc;
}

// Whether [a, a + n) and [b, b + m) share a byte.
inline bool overlap(const void *a, int64_t n, const void *b, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace sv
