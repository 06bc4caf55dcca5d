// Attention of few query rows over the 4-bit cache: decoded tokens, a few drafted ones.
#pragma once

#include "attn_q4.h"
#include "q4.cuh"

namespace kda {

constexpr int F4_KEYS = 32;            // keys a chunk: what a warp loads and works on at a time
constexpr long long F4_MAX_KEYS = 0x7fffff00;
constexpr int F4_SHARE = 4;            // chunks a CTA has at least
constexpr int F4_MAX_CTAS = 160;
constexpr int F4_MAX_ROWS = 16;        // rows a unit can have
constexpr float F4_MOST = 65536.0f;    // sum of a lane's weights that makes a warp look at its maximum

// Rows a unit has at most, and how a CTA is made for them
template <int D, int ROWS>
struct F4Layout {
    static constexpr int WARPS = ROWS == 16 ? 8 : 12;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int STAGES = 2;                              // a warp's ring of chunks
    static constexpr int TILES = ROWS / 8;                        // of 8 queries, the columns of a product
    // A chunk: codes of keys and values, then their scales
    static constexpr uint32_t CODES = F4_KEYS * (D / 2), SCALES = F4_KEYS * (D / 32);
    static constexpr uint32_t STAGE = 2 * (CODES + SCALES);
    static constexpr uint32_t RING = STAGES * STAGE;              // of a warp
    // Partial outputs [row][D] fp32: of the unit that a warp's share begins in; the one it ends in takes the ring's place
    static constexpr uint32_t PART = WARPS * RING;
    static constexpr uint32_t PART_ROW = D * 4, PART_WARP = ROWS * PART_ROW;
    static constexpr uint32_t ML = PART + WARPS * PART_WARP;      // [warp][begin, end][row] reference, sum
    static constexpr uint32_t BYTES = ML + WARPS * 2 * ROWS * 8 + 128;
    static_assert(PART_WARP <= RING, "a partial output in the ring's place");
    static_assert(BYTES <= 232448, "few-row attention shared memory");
};

struct F4Join {
    int n, hk, row0, rows, pieces;   // request, head, first row of the unit among the request's, rows, CTAs
};

struct F4Params {
    AttnQ4Args a;
    F4Join *join;
    float2 *ml;       // [CTA][2][F4_MAX_ROWS]
    float *o;         // [CTA][2][F4_MAX_ROWS][D]
    float c;          // scale log2(e)
    int G;
    uint32_t over_g;  // 2^16 / G, rounded up: (row over_g) >> 16 is row / G for the rows of this kernel's requests
    int most_rows;    // requests with more rows are another kernel's
    int unit_cost;    // of a unit, in chunks
    // Constants that the compiler does not know: a product with a power of two stays one (the multiplier has room, the
    // shifter has not), and a mask with a leading bit stays one instruction.
    uint32_t two20, two4, mask_low, bit_low, mask_high, bit_high, bit_bf16;
};

// Token of a request's row (exact: row < 512, G <= 128)
__device__ __forceinline__ int f4_token(const F4Params &p, int row) { return (int)((uint32_t)row * p.over_g >> 16); }

// One request's units
struct F4Request {
    int row0, fresh, keys, rows, units;
    __device__ void load(const F4Params &p, int n, int R) {
        row0 = p.a.cu[n];
        fresh = p.a.cu[n + 1] - row0;
        keys = p.a.lens[n];
        const long long r = (long long)fresh * p.G;
        rows = fresh > 0 && r <= p.most_rows ? (int)r : 0;
        units = (rows + R - 1) / R;
    }
    // keys that the rows up to (not including) row `end` of the request see
    __device__ int seen(const F4Params &p, int end) const { return keys - fresh + f4_token(p, min(end, rows) - 1) + 1; }
    __device__ int chunks(const F4Params &p, int end) const {
        const int s = seen(p, end);
        return s > F4_KEYS ? (s + F4_KEYS - 1) / F4_KEYS : 1;
    }
    __device__ long long length(const F4Params &p, int R) const {   // of one head's units
        long long sum = 0;
        for (int u = 0; u < units; ++u) sum += chunks(p, (u + 1) * R) + p.unit_cost;
        return sum;
    }
};

// The pieces of units in a warp's share
struct F4Walk {
    F4Request r;
    int n, hk, unit, at;
    long long left;
    int a, b, all, first, rows, seen;   // chunks [a, b) of `all`; the unit's first row and rows; keys its last row sees
    long long rest;                     // of the unit's line after the share
    __device__ bool next(const F4Params &p, int R) {
        for (;;) {
            if (left <= 0) return false;
            if (unit >= r.units) {
                unit = 0;
                if (++hk == p.a.H_kv) {
                    hk = 0;
                    do r.load(p, ++n, R);
                    while (r.units == 0);
                }
            }
            first = unit * R;
            rows = min(R, r.rows - first);
            seen = r.seen(p, first + R);
            all = r.chunks(p, first + R);
            const int whole = all + p.unit_cost, from = at;
            const long long end = at + left;
            const int to = end >= whole ? whole : (int)end;
            left = end - to;
            rest = whole - to;
            a = max(from - p.unit_cost, 0);
            b = max(to - p.unit_cost, 0);
            at = 0;
            ++unit;
            if (b > a) return true;
        }
    }
};

// What a warp has of a unit that its share cuts
struct F4Part {
    int n, hk, first, rows;
    bool there, ends;   // whether there is one, whether it holds the unit's last chunk
    long long rest;     // of the unit's line behind it
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// lo, hi as fp16, rounded to nearest
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

}  // namespace kda
