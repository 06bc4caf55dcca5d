// Arguments of the softmax-attention kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

struct AttnArgs {
    const uint16_t *q, *k, *v;   // k, v: [B, T, H_kv, D], or the caches [num_blocks, H_kv, block, D]
    uint16_t *out;
    float *lse;                  // NULL: not written
    const int32_t *cu;           // NULL: B prompts of T tokens
    const int32_t *table, *lens; // lens NULL: whole prompts
    float scale;
    int N, B, T, H_q, H_kv, D;
    int num_blocks, block_log2, max_blocks;
};

// Whether the call needs its workspace, and the size of one for any lengths.
bool attn_may_cut(const AttnArgs &a);
size_t attn_workspace_bytes(int D);
cudaError_t launch_attn(const AttnArgs &a, void *ws, cudaStream_t stream, int *launches);   // adds to *launches

}  // namespace kda
