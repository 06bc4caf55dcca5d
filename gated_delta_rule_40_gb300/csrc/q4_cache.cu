// The paged key/value cache held in 4 bits: the quantising store of new keys and values, and rows read back.
#include "attn_q4.h"
#include "q4.cuh"

namespace kda {
namespace {

constexpr int Q4_THREADS = 256;

// Byte offsets of a row's codes and scales in a cache
struct Q4Place {
    size_t codes, scales;
};
template <int D>
__device__ __forceinline__ Q4Place q4_place(long long slot, int h, int H_kv, int block_log2) {
    const long long blk = slot >> block_log2, off = slot & ((1ll << block_log2) - 1);
    const size_t base = ((size_t)(blk * H_kv + h) << block_log2) * q4_row_bytes(D);
    return {base + (size_t)off * q4_code_bytes(D),
            base + ((size_t)q4_code_bytes(D) << block_log2) + (size_t)off * q4_scale_bytes(D)};
}

// One word of 8 channels, as codes under the common scale of the four lanes that hold a block of 32
__device__ __forceinline__ uint32_t quantise(const uint4 &u, uint32_t *scale) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float x[8], most = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
        most = fmaxf(most, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
    }
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
    const uint32_t b = q4_scale_byte(most);
    const float inv = __frcp_rn(q4_scale(b));
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) word |= q4_code(x[c], inv) << q4_bit(c);
    *scale = b;
    return word;
}

// The scale bytes of a row, gathered in the row's first lane (a block of 32 is four lanes)
template <int D>
__device__ __forceinline__ uint32_t gather_scales(uint32_t b, int lane) {
    uint32_t all = b;
#pragma unroll
    for (int i = 1; i < D / 32; ++i) all |= __shfl_down_sync(0xffffffffu, b, 4 * i) << (8 * i);
    return all;
}
template <int D>
__device__ __forceinline__ void store_scales(uint8_t *at, uint32_t all) {
    if (D == 128) *reinterpret_cast<uint32_t *>(at) = all;
    else *reinterpret_cast<uint16_t *>(at) = (uint16_t)all;
}

// A lane takes one word of a (token, head) of k and the same one of v.
template <int D>
__global__ __launch_bounds__(Q4_THREADS) void kv_write_q4_kernel(const Q4CacheArgs p, long long units) {
    constexpr int L = D / 8;
    const long long u = (long long)blockIdx.x * Q4_THREADS + threadIdx.x;
    const int lane = threadIdx.x & 31;
    const bool on = u < units;
    const long long row = on ? u / L : 0, t = row / p.H_kv;
    const int x = (int)(u % L), h = (int)(row - t * p.H_kv);
    const long long slot = on ? p.slots[t] : -1;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (on) {
        a = __ldcs(reinterpret_cast<const uint4 *>(p.k + t * p.k_stride + h * D) + x);
        b = __ldcs(reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + h * D) + x);
    }
    uint32_t sk, sv;
    const uint32_t wk = quantise(a, &sk), wv = quantise(b, &sv);
    const uint32_t ak = gather_scales<D>(sk, lane), av = gather_scales<D>(sv, lane);
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        set_status(KDA_ERR_BAD_PAGES);
        return;
    }
    const Q4Place at = q4_place<D>(slot, h, p.H_kv, p.block_log2);
    reinterpret_cast<uint32_t *>(p.k_cache + at.codes)[x] = wk;
    reinterpret_cast<uint32_t *>(p.v_cache + at.codes)[x] = wv;
    if (x == 0) {
        store_scales<D>(p.k_cache + at.scales, ak);
        store_scales<D>(p.v_cache + at.scales, av);
    }
}

// Word x of a row as 8 bf16 values
template <int D>
__device__ __forceinline__ uint4 values_of(uint32_t word, uint32_t b) {
    const uint32_t s2 = q4_scale2(b * 0x00010001u), o2 = q4_offset2(s2);
    return make_uint4(q4_value(q4_raw(word, 0), s2, o2), q4_value(q4_raw(word, 1), s2, o2),
                      q4_value(q4_raw(word, 2), s2, o2), q4_value(q4_raw(word, 3), s2, o2));
}

template <int D>
__global__ __launch_bounds__(Q4_THREADS) void kv_read_q4_kernel(const Q4CacheArgs p, long long units) {
    constexpr int L = D / 8;
    const long long u = (long long)blockIdx.x * Q4_THREADS + threadIdx.x;
    if (u >= units) return;
    const long long row = u / L, t = row / p.H_kv;
    const int x = (int)(u % L), h = (int)(row - t * p.H_kv);
    const long long slot = p.slots[t];
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (slot >= p.num_slots) set_status(KDA_ERR_BAD_PAGES);
    if (slot >= 0 && slot < p.num_slots) {
        const Q4Place at = q4_place<D>(slot, h, p.H_kv, p.block_log2);
        const uint32_t wk = reinterpret_cast<const uint32_t *>(p.k_cache + at.codes)[x];
        const uint32_t wv = reinterpret_cast<const uint32_t *>(p.v_cache + at.codes)[x];
        a = values_of<D>(wk, p.k_cache[at.scales + x / 4]);
        b = values_of<D>(wv, p.v_cache[at.scales + x / 4]);
    }
    __stcs(reinterpret_cast<uint4 *>(p.k_out) + u, a);
    __stcs(reinterpret_cast<uint4 *>(p.v_out) + u, b);
}
}  // namespace

cudaError_t launch_kv_write_q4(const Q4CacheArgs &a, cudaStream_t stream) {
    const long long units = (long long)a.T * a.H_kv * (a.D / 8);
    const unsigned grid = (unsigned)((units + Q4_THREADS - 1) / Q4_THREADS);
    if (a.D == 64) kv_write_q4_kernel<64><<<grid, Q4_THREADS, 0, stream>>>(a, units);
    else kv_write_q4_kernel<128><<<grid, Q4_THREADS, 0, stream>>>(a, units);
    return cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const Q4CacheArgs &a, cudaStream_t stream) {
    const long long units = (long long)a.T * a.H_kv * (a.D / 8);
    const unsigned grid = (unsigned)((units + Q4_THREADS - 1) / Q4_THREADS);
    if (a.D == 64) kv_read_q4_kernel<64><<<grid, Q4_THREADS, 0, stream>>>(a, units);
    else kv_read_q4_kernel<128><<<grid, Q4_THREADS, 0, stream>>>(a, units);
    return cudaGetLastError();
}

}  // namespace kda
