// Causal softmax attention over a paged cache held in 4 bits (kda_attn_paged_q4): a warp a (token, head).
#include "attn_q4.h"
#include "q4.cuh"

namespace kda {
size_t attn_q4_few_workspace_bytes(int D);
cudaError_t launch_attn_q4_few(const AttnQ4Args &a, int most_rows, void *ws, cudaStream_t stream, int *launches);

namespace {
// Rows (new tokens x query heads of a group) of a request up to which the kernel for few rows takes it
constexpr int F4_MOST_ROWS = 32;

template <int D>
__global__ __launch_bounds__(256) void attn_q4_simple_kernel(const AttnQ4Args p) {
    constexpr int CODES = q4_code_bytes(D), SCALES = q4_scale_bytes(D);
    __shared__ float s_q[8][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = p.cu[0] != 0 || p.cu[p.N] > p.T;
    for (int n = threadIdx.x; n < p.N; n += 256)
        bad |= p.cu[n + 1] < p.cu[n] || p.lens[n] < 0 || p.lens[n] > ((long long)p.max_blocks << p.block_log2);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_status(KDA_ERR_BAD_SEQLENS);
        return;
    }
    const long long item = (long long)blockIdx.x * 8 + warp;
    const long long t = item / p.H_q;
    if (t >= p.cu[p.N]) return;
    const int h = (int)(item - t * p.H_q), hk = h / (p.H_q / p.H_kv);
    int lo = 0, hi = p.N;   // the last request that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    if ((long long)(p.cu[lo + 1] - p.cu[lo]) * (p.H_q / p.H_kv) <= F4_MOST_ROWS) return;   // the other kernel's
    const int limit = p.lens[lo] - (p.cu[lo + 1] - (int)t) + 1;   // keys seen
    const size_t row = (size_t)t * p.H_q + h;
    for (int d = lane; d < D; d += 32) s_q[warp][d] = bf16_to_f(p.q[row * D + d]) * p.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    const int bs = 1 << p.block_log2;
    for (int j0 = 0; j0 < limit; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        int id = -1;
        if (j < limit) {
            id = p.table[(size_t)lo * p.max_blocks + (j >> p.block_log2)];
            s = 0.f;
            if (id < 0 || id >= p.num_blocks) {
                set_status(KDA_ERR_BAD_PAGES);
                id = -1;
            } else {
                const uint8_t *base = p.k + (((size_t)id * p.H_kv + hk) << p.block_log2) * (CODES + SCALES);
                const uint32_t *c = reinterpret_cast<const uint32_t *>(base + (size_t)(j & (bs - 1)) * CODES);
                const uint8_t *sc = base + (size_t)bs * CODES + (size_t)(j & (bs - 1)) * SCALES;
                for (int w = 0; w < D / 8; ++w) {
                    const uint32_t word = c[w];
                    float part = 0.f;
                    for (int i = 0; i < 8; ++i) part += ((int)(word >> q4_bit(i) & 15u) - 8) * s_q[warp][8 * w + i];
                    s += part * q4_scale(sc[w / 4]);
                }
            }
        }
        float top = s;
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float next = fmaxf(m, top), ref = next == -INFINITY ? 0.f : next;
        const float f = __expf(m - ref), pj = __expf(s - ref);
        l = l * f + warp_sum(pj);
        m = next;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] *= f;
        for (int k = 0; k < 32; ++k) {
            const float pk = __shfl_sync(0xffffffffu, pj, k);
            const int idk = __shfl_sync(0xffffffffu, id, k);
            if (idk < 0) continue;
            const int in = (j0 + k) & (bs - 1);
            const uint8_t *base = p.v + (((size_t)idk * p.H_kv + hk) << p.block_log2) * (CODES + SCALES);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = 32 * i + lane;
                const uint32_t word = reinterpret_cast<const uint32_t *>(base + (size_t)in * CODES)[d / 8];
                o[i] += pk * ((int)(word >> q4_bit(d & 7) & 15u) - 8) * q4_scale(base[(size_t)bs * CODES + in * SCALES + i]);
            }
        }
    }
    const float inv = limit > 0 ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) p.out[row * D + 32 * i + lane] = limit > 0 ? f_to_bf16(o[i] * inv) : 0;
    if (lane == 0 && p.lse) p.lse[row] = limit > 0 ? m + logf(l) : -INFINITY;
}
}  // namespace

size_t attn_q4_workspace_bytes(int D) { return attn_q4_few_workspace_bytes(D); }

cudaError_t launch_attn_q4(const AttnQ4Args &a, void *ws, cudaStream_t stream, int *launches) {
    cudaError_t e = launch_attn_q4_few(a, F4_MOST_ROWS, ws, stream, launches);
    if (e != cudaSuccess || (long long)a.T * (a.H_q / a.H_kv) <= F4_MOST_ROWS) return e;
    const unsigned grid = (unsigned)(((long long)a.T * a.H_q + 7) / 8);
    ++*launches;
    if (a.D == 64) attn_q4_simple_kernel<64><<<grid, 256, 0, stream>>>(a);
    else attn_q4_simple_kernel<128><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
