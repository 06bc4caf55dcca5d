// The paged key/value cache held in 4 bits: the quantising store of new keys and values, and rows read back.
//
// Both are one pass over rows, lanes on neighbouring 32 (store) or 16 (read) bytes, codes and bf16 rows in whole
// sectors.  On the GPU, 32768 tokens x 8 heads of 128, back to back: store 28 us, 6.0 TB/s (with one word a lane, and
// rounding by conversions to integers, 52 us; with five instead of six blocks an SM 28.9 us); read 27.4 us, 6.2 TB/s
// (one row a lane 32.6, four 28.1; blocks of 256 threads 30.2 us).  64 tokens: 2 us each.
#include "attn_q4.h"
#include "q4.cuh"

namespace kda {
namespace {

constexpr int Q4_THREADS = 256;
constexpr int Q4_READ_THREADS = 128, Q4_READS = 2;   // rows that a lane reads

// Byte offsets of a row's codes and scales in a cache
struct Q4Place {
    size_t codes, scales;
};
template <int D>
__device__ __forceinline__ Q4Place q4_place(long long slot, uint32_t h, int H_kv, int block_log2) {
    const long long blk = slot >> block_log2, off = slot & ((1ll << block_log2) - 1);
    const size_t base = ((size_t)(blk * H_kv + h) << block_log2) * q4_row_bytes(D);
    return {base + (size_t)off * q4_code_bytes(D),
            base + ((size_t)q4_code_bytes(D) << block_log2) + (size_t)off * q4_scale_bytes(D)};
}

// Largest magnitude among the 32 channels that two lanes hold, as bf16 bits: magnitudes order as integers
__device__ __forceinline__ uint32_t largest(const uint4 (&u)[2]) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        x = __vimax3_u16x2(__vimax3_u16x2(x, u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu), u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu);
    const uint32_t m = max(x & 0xffffu, x >> 16);
    return max(m, __shfl_xor_sync(0xffffffffu, m, 1));
}

// A word's codes under scale s.  They are rounded by adding 1.5 2^23 and packed four at a time by products with powers of
// 16, all exact, as the multiplier has room and the shifter has not: channels 2j in one half, 2j + 1 in the other.
__device__ __forceinline__ uint32_t codes_of(const uint4 &u, float s, float inv, bool clamp) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    constexpr float ROUND = 12582912.f;
    float2 sum = make_float2(ROUND + (float)0x8888, ROUND + (float)0x8888);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 x = make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
        if (clamp) {   // numbers past the largest scale's range
            x.x = fminf(fmaxf(x.x, -7.f * s), 7.f * s);
            x.y = fminf(fmaxf(x.y, -7.f * s), 7.f * s);
        }
        x = __fadd2_rn(__ffma2_rn(x, make_float2(inv, inv), make_float2(ROUND, ROUND)), make_float2(-ROUND, -ROUND));
        sum = __ffma2_rn(x, make_float2((float)(1 << 4 * j), (float)(1 << 4 * j)), sum);
    }
    return __byte_perm(__float_as_uint(sum.x), __float_as_uint(sum.y), 0x5410);
}

// NaNs become 0
__device__ __forceinline__ uint32_t no_nan(uint32_t w) {
    if ((w & 0x7fffu) > 0x7f80u) w &= 0xffff0000u;
    if ((w >> 16 & 0x7fffu) > 0x7f80u) w &= 0xffffu;
    return w;
}

}  // namespace

// A lane takes 16 channels of a (token, head) of k and the same ones of v: two words, half a block of 32.
template <int D>
__global__ __launch_bounds__(Q4_THREADS, 6) void kv_write_q4_kernel(const Q4CacheArgs p, uint32_t rows) {
    constexpr uint32_t L = D / 16;
    const uint32_t row = blockIdx.x * (Q4_THREADS / L) + threadIdx.x / L, x = threadIdx.x % L;
    const bool on = row < rows;
    const uint32_t t = on ? row / (uint32_t)p.H_kv : 0, h = row - t * (uint32_t)p.H_kv;
    const long long slot = on ? p.slots[t] : -1;
    uint4 u[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        u[0][i] = u[1][i] = make_uint4(0, 0, 0, 0);
        if (on) {
            u[0][i] = __ldcs(reinterpret_cast<const uint4 *>(p.k + t * p.k_stride + h * D) + 2 * x + i);
            u[1][i] = __ldcs(reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + h * D) + 2 * x + i);
        }
    }
    uint32_t most[2] = {largest(u[0]), largest(u[1])}, scale[2], word[2][2];
    bool rare = max(most[0], most[1]) >= 0x7f80u;
    if (__any_sync(0xffffffffu, rare)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                u[i][j] = make_uint4(no_nan(u[i][j].x), no_nan(u[i][j].y), no_nan(u[i][j].z), no_nan(u[i][j].w));
            most[i] = largest(u[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) scale[i] = q4_scale_byte(__uint_as_float(most[i] << 16));
    rare = max(scale[0], scale[1]) == 255;
    rare = __any_sync(0xffffffffu, rare);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float s = q4_scale(scale[i]), inv = q4_inverse(s);
        if (rare) {
            word[i][0] = codes_of(u[i][0], s, inv, true);
            word[i][1] = codes_of(u[i][1], s, inv, true);
        } else {
            word[i][0] = codes_of(u[i][0], s, inv, false);
            word[i][1] = codes_of(u[i][1], s, inv, false);
        }
    }
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        set_status(KDA_ERR_BAD_PAGES);
        return;
    }
    const Q4Place at = q4_place<D>(slot, h, p.H_kv, p.block_log2);
    reinterpret_cast<uint2 *>(p.k_cache + at.codes)[x] = make_uint2(word[0][0], word[0][1]);
    reinterpret_cast<uint2 *>(p.v_cache + at.codes)[x] = make_uint2(word[1][0], word[1][1]);
    if ((x & 1) == 0) {
        p.k_cache[at.scales + x / 2] = (uint8_t)scale[0];
        p.v_cache[at.scales + x / 2] = (uint8_t)scale[1];
    }
}

namespace {
// Word x of a row as 8 bf16 values
__device__ __forceinline__ uint4 values_of(uint32_t word, uint32_t b) {
    const Q4Scale s = q4_scales(b * 0x00010001u, 16u);
    auto pair = [&](int j) { return q4_fma(q4_pair(word, j, s), 0x4b004b00u, 0u); };   // 2^23
    return make_uint4(pair(0), pair(1), pair(2), pair(3));
}

}  // namespace

// A lane takes 8 channels of Q4_READS rows, whose loads are in flight together.
template <int D>
__global__ __launch_bounds__(Q4_READ_THREADS) void kv_read_q4_kernel(const Q4CacheArgs p, uint32_t rows) {
    constexpr uint32_t L = D / 8, STEP = Q4_READ_THREADS / L;
    const uint32_t row0 = blockIdx.x * (Q4_READS * STEP) + threadIdx.x / L, x = threadIdx.x % L;
    long long slot[Q4_READS];
    uint32_t head[Q4_READS], k[Q4_READS], v[Q4_READS], ks[Q4_READS], vs[Q4_READS];
#pragma unroll
    for (int i = 0; i < Q4_READS; ++i) {
        const uint32_t row = row0 + i * STEP, t = row / (uint32_t)p.H_kv;
        head[i] = row - t * (uint32_t)p.H_kv;
        slot[i] = row < rows ? p.slots[t] : -1;
        if (slot[i] >= p.num_slots) {
            set_status(KDA_ERR_BAD_PAGES);
            slot[i] = -1;
        }
    }
#pragma unroll
    for (int i = 0; i < Q4_READS; ++i) {
        k[i] = v[i] = 0x88888888u;   // zeros
        ks[i] = vs[i] = 0;
        if (slot[i] < 0) continue;
        const Q4Place at = q4_place<D>(slot[i], head[i], p.H_kv, p.block_log2);
        k[i] = reinterpret_cast<const uint32_t *>(p.k_cache + at.codes)[x];
        v[i] = reinterpret_cast<const uint32_t *>(p.v_cache + at.codes)[x];
        ks[i] = p.k_cache[at.scales + x / 4];
        vs[i] = p.v_cache[at.scales + x / 4];
    }
#pragma unroll
    for (int i = 0; i < Q4_READS; ++i) {
        const uint32_t row = row0 + i * STEP;
        if (row >= rows) continue;
        __stcs(reinterpret_cast<uint4 *>(p.k_out) + (size_t)row * L + x, values_of(k[i], ks[i]));
        __stcs(reinterpret_cast<uint4 *>(p.v_out) + (size_t)row * L + x, values_of(v[i], vs[i]));
    }
}

namespace {
// Blocks of `threads` lanes that take `channels` of `each` rows
unsigned grid_of(const Q4CacheArgs &a, int threads, int channels, int each) {
    const unsigned rows = threads / (a.D / channels) * each;   // a block
    return (unsigned)(((long long)a.T * a.H_kv + rows - 1) / rows);
}
}  // namespace

cudaError_t launch_kv_write_q4(const Q4CacheArgs &a, cudaStream_t stream) {
    const uint32_t rows = (uint32_t)a.T * (uint32_t)a.H_kv;   // below 2^31, as the entry point checks
    if (a.D == 64) kv_write_q4_kernel<64><<<grid_of(a, Q4_THREADS, 16, 1), Q4_THREADS, 0, stream>>>(a, rows);
    else kv_write_q4_kernel<128><<<grid_of(a, Q4_THREADS, 16, 1), Q4_THREADS, 0, stream>>>(a, rows);
    return cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const Q4CacheArgs &a, cudaStream_t stream) {
    const uint32_t rows = (uint32_t)a.T * (uint32_t)a.H_kv;
    if (a.D == 64) kv_read_q4_kernel<64><<<grid_of(a, Q4_READ_THREADS, 8, Q4_READS), Q4_READ_THREADS, 0, stream>>>(a, rows);
    else kv_read_q4_kernel<128><<<grid_of(a, Q4_READ_THREADS, 8, Q4_READS), Q4_READ_THREADS, 0, stream>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace kda
