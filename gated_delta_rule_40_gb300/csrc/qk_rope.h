// Arguments of the query/key norm and rotation kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

struct QkRopeArgs {
    const uint16_t *q, *k;           // [T, H, D], tokens q_stride and k_stride elements apart
    long long q_stride, k_stride;
    const float *q_weight, *k_weight;   // NULL: ones
    float eps;
    int norm;                        // 0: rotation only
    const float *freqs;              // [rot / 2] radians a token
    int rot, interleaved;
    const int32_t *positions;        // negative: the token is left out
    int T, H_q, H_kv, D;
    uint16_t *q_out, *k_out;         // forward
    const uint16_t *dq_out, *dk_out; // backward
    float *dq, *dk, *dq_weight, *dk_weight;
};

cudaError_t launch_qk_rope(const QkRopeArgs &a, cudaStream_t stream);
size_t qk_rope_bwd_workspace_bytes(int D);
cudaError_t launch_qk_rope_bwd(const QkRopeArgs &a, void *ws, cudaStream_t stream, int *launches);

}  // namespace kda
