// Attention of few query rows over the 4-bit cache: decoded tokens, a few drafted ones.
#pragma once

#include "attn_q4.h"
#include "q4.cuh"

namespace kda {

constexpr int F4_KEYS = 32;            // keys a chunk: what a warp loads and works on at a time
constexpr long long F4_MAX_KEYS = 0x7fffff00;
// Chunks a CTA has at least (a token over 1000 keys, 8 heads: 4 10.6 us, 1 11.2, 12 11.3, 24 12.7; four such: 10.9, 10.9,
// 11.4, 12.8)
constexpr int F4_SHARE = 4;
constexpr int F4_MAX_ROWS = 16;        // rows a unit can have
constexpr float F4_MOST = 65536.f * Q4_UP;   // sum of a lane's weights (2^23 for 1) that makes a warp look at its maximum

// Rows a unit has at most, and how a CTA is made for them
template <int D, int ROWS>
struct F4Layout {
    static constexpr int WARPS = ROWS == 16 && D == 128 ? 8 : 12;   // by registers
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
    // Powers of two that the compiler does not know, so that products with them stay products: the multiplier has room, the
    // shifter has not
    uint32_t two20, two4;
};

// Token of a request's row (exact: row < 512, G <= 128)
__device__ __forceinline__ int f4_token(const F4Params &p, int row) { return (int)((uint32_t)row * p.over_g >> 16); }

// One request's units
struct F4Request {
    int row0, fresh, keys, rows, units;
    __device__ void load(const F4Params &p, int n, int R) {
        row0 = p.a.cu[n];
        fresh = (int)((uint32_t)p.a.cu[n + 1] - (uint32_t)row0);   // (offsets that fall are found by comparing them)
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

// Joins the pieces of a unit that several CTAs worked on, in the order of the CTAs.
// Thread i of D / 4 for each row.
template <int D>
__device__ __forceinline__ void f4_join(const F4Params &p, int cta, int i) {
    const F4Join d = p.join[cta];
    const int row = i / (D / 4), piece = i % (D / 4);
    if (d.pieces == 0 || row >= d.rows) return;
    auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * cta + 1 : 2 * (cta + k)); };
    float M = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < d.pieces; k0 += 4) {   // four at a time, so that their loads are in flight together
        float2 ml[4];
        float4 x[4];
        float top = M;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + k < d.pieces) {
                ml[k] = p.ml[slot(k0 + k) * F4_MAX_ROWS + row];
                x[k] = *reinterpret_cast<const float4 *>(p.o + (slot(k0 + k) * F4_MAX_ROWS + row) * D + 4 * piece);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
        const float ref = top == -INFINITY ? 0.f : top, f0 = ex2(M - ref);
        l *= f0;
        o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
        M = top;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = ex2(ml[k].x - ref);
            l += f * ml[k].y;
            o.x += f * x[k].x; o.y += f * x[k].y; o.z += f * x[k].z; o.w += f * x[k].w;
        }
    }
    const int row0 = p.a.cu[d.n], fresh = p.a.cu[d.n + 1] - row0, flat = d.row0 + row, tok = flat / p.G;
    const size_t at = (size_t)(row0 + tok) * p.a.H_q + d.hk * p.G + (flat - tok * p.G);
    if (p.a.lens[d.n] - fresh + tok + 1 <= 0) l = 0.f;
    const float inv = l != 0.f ? 1.f / l : 0.f, ref = M == -INFINITY ? 0.f : M;
    *reinterpret_cast<uint2 *>(p.a.out + at * D + 4 * piece) =
        l == 0.f ? make_uint2(0, 0) : make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (piece == 0 && p.a.lse) p.a.lse[at] = l == 0.f ? -INFINITY : (ref + lg2(l)) * (1.f / LOG2E);
}

int attn_q4_few_rows(const AttnQ4Args &a, int most_rows);   // of a unit
F4Params attn_q4_few_params(const AttnQ4Args &a, int most_rows, void *ws);
size_t attn_q4_few_workspace_bytes(int D);
// The kernel for few rows, and the joining of its pieces where no kernel for chunks follows
cudaError_t launch_attn_q4_few(const F4Params &p, int rows, cudaStream_t stream, int *launches);
cudaError_t launch_attn_q4_few_join(const F4Params &p, int rows, cudaStream_t stream, int *launches);
// Attention of the requests with more than few_tokens new tokens (k and v of `a` point to the cache's bytes).  Where the
// kernel for the others is the stream's latest, `few` has its arguments, and its pieces are joined together with this
// one's; NULL: none was launched.
struct AttnArgs;
cudaError_t launch_attn_q4_many(const AttnArgs &a, int few_tokens, const F4Params *few, int few_rows, void *ws,
                                cudaStream_t stream, int *launches);

}  // namespace kda
