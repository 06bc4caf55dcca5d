// Arguments of the kernels of the 4-bit cache.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

struct Q4CacheArgs {
    const uint16_t *k, *v;        // store: [T, H_kv, D], tokens k_stride and v_stride elements apart
    long long k_stride, v_stride;
    uint16_t *k_out, *v_out;      // read: [T, H_kv, D]
    const int32_t *slots;
    uint8_t *k_cache, *v_cache;   // [num_blocks, H_kv, block, D / 2 + D / 32]
    int T, H_kv, D, block_log2;
    long long num_slots;
};

cudaError_t launch_kv_write_q4(const Q4CacheArgs &a, cudaStream_t stream);
cudaError_t launch_kv_read_q4(const Q4CacheArgs &a, cudaStream_t stream);

struct AttnQ4Args {
    const uint16_t *q;
    const uint8_t *k, *v;         // the caches
    uint16_t *out;
    float *lse;                   // NULL: not written
    const int32_t *cu, *table, *lens;
    float scale;
    int N, T, H_q, H_kv, D;
    int num_blocks, block_log2, max_blocks;
};

size_t attn_q4_workspace_bytes(int D);
cudaError_t launch_attn_q4(const AttnQ4Args &a, void *ws, cudaStream_t stream, int *launches);

}  // namespace kda
