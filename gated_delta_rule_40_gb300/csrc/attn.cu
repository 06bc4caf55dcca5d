// Causal softmax attention with grouped heads, over whole prompts (kda_attn_fwd) and over a paged
// cache (kda_attn_paged): s = scale q.k, o = sum exp(s - lse) v over the keys up to the query's own.
#include "kda_common.cuh"
#include "attn.h"

namespace kda {

// One warp a (token, query head).  Lane l holds channels l, l + 32, ... of q and of the output; the
// running maximum and sum of the softmax are rescaled when the maximum grows.
template <int D, bool PAGED>
__global__ __launch_bounds__(256) void attn_row_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    // every warp checks the lengths, so that a malformed call writes nothing
    const int nseq = a.cu ? a.N : a.B;
    bool ok = true;
    if (a.cu) {
        for (int n = lane; n < a.N; n += 32) {
            ok &= a.cu[n + 1] >= a.cu[n];
            if (PAGED) ok &= a.lens[n] >= 0 && a.lens[n] <= ((long long)a.max_blocks << a.block_log2);
        }
        ok &= a.cu[0] == 0 && (PAGED ? a.cu[a.N] <= a.T : a.cu[a.N] == a.T);
    }
    if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) set_status(KDA_ERR_BAD_SEQLENS);
        return;
    }
    const long long tokens = (long long)a.B * a.T;
    if (row >= tokens * a.H_q) return;
    const long long t = row / a.H_q;
    const int h = (int)(row - t * a.H_q), hk = h / (a.H_q / a.H_kv);
    int n = 0;
    long long first, keys;   // first key row (prompts), number of keys seen
    if (a.cu) {
        while (n < nseq && a.cu[n + 1] <= t) ++n;
        if (n >= nseq) return;
        first = a.cu[n];
        keys = t - first + 1;
        if (PAGED) keys += a.lens[n] - (a.cu[n + 1] - a.cu[n]);
    } else {
        n = (int)(t / a.T);
        first = (long long)n * a.T;
        keys = t - first + 1;
    }
    constexpr int R = D / 32;
    float q[R], o[R], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        q[i] = bf16_to_f(a.q[row * D + lane + 32 * i]) * (a.scale * LOG2E);
        o[i] = 0.f;
    }
    for (long long j = 0; j < keys; ++j) {
        long long at;
        bool real = true;
        if (PAGED) {
            const int id = a.table[(size_t)n * a.max_blocks + (j >> a.block_log2)];
            real = id >= 0 && id < a.num_blocks;
            if (!real && lane == 0) set_status(KDA_ERR_BAD_PAGES);
            at = ((((long long)id * a.H_kv + hk) << a.block_log2) + (j & ((1 << a.block_log2) - 1))) * D;
        } else {
            at = ((first + j) * a.H_kv + hk) * D;
        }
        float s = 0.f;
        if (real) {
#pragma unroll
            for (int i = 0; i < R; ++i) s += q[i] * bf16_to_f(a.k[at + lane + 32 * i]);
        }
        s = warp_sum(s);
        const float m2 = fmaxf(m, s), c = ex2(m - m2), e = ex2(s - m2);
        l = l * c + e;
#pragma unroll
        for (int i = 0; i < R; ++i) o[i] = o[i] * c + (real ? e * bf16_to_f(a.v[at + lane + 32 * i]) : 0.f);
        m = m2;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) a.out[row * D + lane + 32 * i] = f_to_bf16(o[i] * inv);
    if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + lg2(l)) * (1.f / LOG2E) : -INFINITY;
}

cudaError_t launch_attn(const AttnArgs &a, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.T * a.H_q;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (a.lens)
        a.D == 64 ? attn_row_kernel<64, true><<<grid, 256, 0, stream>>>(a)
                  : attn_row_kernel<128, true><<<grid, 256, 0, stream>>>(a);
    else
        a.D == 64 ? attn_row_kernel<64, false><<<grid, 256, 0, stream>>>(a)
                  : attn_row_kernel<128, false><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
