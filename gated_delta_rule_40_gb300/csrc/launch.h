// What the launchers of the softmax layers' operators share.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

namespace kda {

constexpr int MAX_SMS = 160;   // that a launch is made for, and workspaces

// SMs of the current device, at most MAX_SMS; 0 where there is none
inline int sm_count() {
    static int count[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!count[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        count[dev] = n < MAX_SMS ? n : MAX_SMS;
    }
    return count[dev];
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace kda
