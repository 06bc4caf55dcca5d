// Attention of few query rows over the 4-bit cache: decoded tokens, a few drafted ones.
#pragma once

#include "attn_q4.h"
#include "kda_tma.cuh"
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
    static constexpr int WARPS = ROWS == 16 ? 7 : 15;           // that attend; one more loads
    static constexpr int THREADS = 32 * (WARPS + 1);
    static constexpr int STAGES = ROWS == 16 ? 4 : 2;                             // a warp's ring
    static constexpr int TILES = ROWS / 4;                        // score tiles: 4 queries, each a high and a low column
    static constexpr int QT = (ROWS + 7) / 8;                     // output tiles of 8 columns
    static constexpr uint32_t CODES = F4_KEYS * (D / 2), SCALES = F4_KEYS * (D / 32);
    static constexpr uint32_t STAGE = 2 * CODES;                  // of codes: keys, then values
    static constexpr uint32_t RING = WARPS * STAGES * STAGE;
    static constexpr uint32_t SC = RING, SC_STAGE = 2 * SCALES;
    static constexpr uint32_t PART = SC + WARPS * STAGES * SC_STAGE;   // partial outputs [buffer][warp][row][D] fp32
    static constexpr int BUFS = ROWS == 4 ? 2 : 1;
    static constexpr uint32_t PART_ROW = D * 4;
    static constexpr uint32_t PART_WARP = ROWS * PART_ROW;
    static constexpr uint32_t ML = PART + BUFS * WARPS * PART_WARP;    // [buffer][warp][row] reference, sum
    static constexpr uint32_t BAR = ML + BUFS * WARPS * ROWS * 8;
    // barriers: chunk loaded / free [warp][stage], partial outputs written / read [buffer]
    enum { FULL = 0, EMPTY = FULL + WARPS * STAGES, PF = EMPTY + WARPS * STAGES, PE = PF + BUFS, COUNT = PE + BUFS };
    static constexpr uint32_t BADS = BAR + 8 * COUNT;             // [warp][stage] halves of a chunk without a block
    static constexpr uint32_t FLAG = BADS + 4 * WARPS * STAGES;
    static constexpr uint32_t BYTES = FLAG + 16 + 1024;
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
    int most_rows;    // requests with more rows are another kernel's
    int unit_cost;    // of a unit, in chunks
};

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
    __device__ int seen(const F4Params &p, int end) const { return keys - fresh + (min(end, rows) - 1) / p.G + 1; }
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

// The pieces of units in a CTA's share
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

__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2], float c0) {
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c0), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         const uint32_t (&b)[2]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// Two numbers as e4m3, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ float2 e4m3x2_to_f(uint32_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)x));
    float lo, hi;
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}\n" : "=f"(lo), "=f"(hi) : "r"(h));
    return make_float2(lo, hi);
}

}  // namespace kda
