// Attention of few query rows over the 4-bit cache: requests with up to F4_MOST_ROWS (attn_q4.cu) rows, decoded and
// drafted tokens.  s = scale q.k, o = sum exp(s - lse) v over the values that the cache stands for.
//
// Work.  A unit is up to 8 or 16 rows (tokens x query heads of a group) of one (request, key/value head), over the chunks
// of 32 keys that its last row sees.  The chunks of all units, and a constant for each unit's own cost, form one line, cut
// into equal shares: one a warp, so that few units are shared at all.  (With the warps of a CTA all on one unit, every one
// of them pays for every unit's beginning and end: 518 against 166 us for 256 decoded tokens, at the time.)  What a share's
// ends cut is joined in shared memory among a CTA's warps, and among CTAs by attn_q4_join_kernel, or by
// attn_q4_join_both_kernel (attn.cu) where the kernel for chunks runs too, in a fixed order.
//
// A warp by itself, with no barrier until the end: cp.async of a chunk into one of two stages, the next but one in flight
// while it works.  Both products are small ones (mma.sync) with the keys as rows: 16 keys x 16 channels times 8 queries
// for the scores, 16 channels x 16 keys times 8 queries for the outputs, whose operands are expanded from codes in
// registers.  tcgen05, whose rows are 128, would take operands from shared or tensor memory, which costs more here than
// what they compute.
//   scores   codes as fp16 in place, without an exponent (2^-24 c or 2^-20 c), one mask each and one shift a word of 8; q as
//            fp16 times a power of two, which keeps every channel down to 2^-27 of the row's largest (a smaller one is off by
//            2^-35 of that at most); 8 times the sum of q is taken off, and the keys' scale is applied, for each block of
//            32 channels in fp32.  (With an exponent, 1024 + c and 64 + c, the sums are exact to 2^-22 of 1039 instead of
//            15 times the queries' sum: lse was 1e-4 off.)
//   weights  2^(s c - m), c = scale log2(e), with the reference m of the piece's first chunk, which moves when a sum of
//            weights passes 2^16; rounded to bf16 as operands, like attn.cu's
//   outputs  codes of two keys in the halves of a register, as bf16 without an exponent, times the keys' scales less 8 of
//            them: 2^-23 n s, a bf16 number, for weights that are 2^23 times as large.  (With an exponent, 128 + c, whose
//            offset a product of its own takes off: two shifts more a pair of words.)  Values reach to 9e5, which fp16
//            does not hold (tried with bf16 for what it does not: the same time)
// Lanes read what they expand from 16-byte pieces that are exchanged by the row's place, without bank conflicts.
//
// What bounds it, and what it measured on the GPU.  256 decoded tokens with 0.59 GB of cache in 117 us, 5.0 TB/s: expanding
// and multiplying take 107 us by themselves, the loads 100 us (the floor is 87 us).  A chunk costs an SM 227 cycles, where
// its bytes need 190, and 604 instructions, 270 of them on the logic and shift units (135 cycles at their rate) and 32
// products (60).  No unit is at its limit: instructions issue in 62 % of the cycles, the logic unit is busy 55 %, the
// tensor cores 26 %, DRAM 64 % of its peak, and what warps wait for most is their own last instruction (1.43 an issue), with
// three warps a scheduler.  So it is chains of dependent instructions, and their number.  More warps are no way out: 12 of 168
// registers beat 16 of 128 (115.6 against 122.2 us for 128 tokens over 4096 keys; 51.4 against 52.2 with heads of 64,
// which lose no register to memory), and 8 of 255, whose outputs and next scores were interleaved (154 against 136 us at
// the time).  Products that start at the offsets, two additions less in a score's chain (118.8 against 118.0 us), three
// stages, a block's addresses once for its chunks, and shifts as products (more of them for the multiplier, less for
// the shifter) change nothing or cost up to 5 %.
// 8-bit products (e4m3 holds a code as it is) turn their operands into fp16 first on this chip.
// 4 drafted tokens over 131072 keys, 16 rows: 48 us (two warps a scheduler, all that their registers leave room for, issue
// in 45 % of the cycles); 100 decoded tokens with heads of 64 34 us (the smaller chunks' own cost); 4 decoded tokens over
// up to 1000 keys 8.5 us, all latency.
#include "attn_q4_few.cuh"
#include "launch.h"

#include <cfloat>

namespace kda {
namespace {

// Row of out and lse that is row `flat` of a request's rows of one head's group
__device__ __forceinline__ size_t out_row(const F4Params &p, const F4Request &r, int hk, int flat) {
    const int tok = f4_token(p, flat);
    return (size_t)(r.row0 + tok) * p.a.H_q + hk * p.G + (flat - tok * p.G);
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    float4 x;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a));
    return x;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
    float2 x;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(a));
    return x;
}
__device__ __forceinline__ void sts_f4(uint32_t a, float4 x) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w) : "memory");
}
template <int TO, int FROM>
__device__ __forceinline__ void cp16_at(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;\n" ::"r"(to), "l"(from), "n"(TO), "n"(FROM) : "memory");
}
__device__ __forceinline__ void sts_f2(uint32_t a, float2 x) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x.x), "f"(x.y) : "memory");
}

}  // namespace

template <int D, int ROWS>
__global__ __launch_bounds__(F4Layout<D, ROWS>::THREADS, 1) void attn_q4_few_kernel(const __grid_constant__ F4Params p) {
    using L = F4Layout<D, ROWS>;
    constexpr int W = L::WARPS, S = L::STAGES, TILES = L::TILES, MT = D / 16, BLOCKS = D / 32, ROWB = D / 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = aligned_smem<128>(smem_raw);
    const uint32_t sbase = smem_u32(sm);
    __shared__ long long s_warp[W], s_before[L::THREADS];
    __shared__ F4Walk s_ahead[W];
    __shared__ F4Part s_part[W][2];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    grid_dep_launch();

    // ---- this warp's share of the line of all units: a CTA's is cut into as many as it has warps
    F4Walk w = {};
    long long share;   // of a CTA
    {
        if (tid == 0) p.join[blockIdx.x].pieces = 0;
        if (lane < 2) s_part[warp][lane].there = false;
        bool bad = tid == 0 && (p.a.cu[0] != 0 || p.a.cu[p.a.N] > p.a.T);
        const long long most = min((long long)p.a.max_blocks << p.a.block_log2, F4_MAX_KEYS);
        const int per = (p.a.N + L::THREADS - 1) / L::THREADS, n0 = min(tid * per, p.a.N), n1 = min(n0 + per, p.a.N);
        long long mine = 0;
        F4Request r;
        for (int n = n0; n < n1; ++n) {
            r.load(p, n, ROWS);
            // offsets that fall, by more than 2^31 too, which their difference does not show
            if (p.a.cu[n + 1] < r.row0 || r.keys < 0 || r.keys > most) bad = true;
            else mine += r.length(p, ROWS) * p.a.H_kv;
        }
        long long before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        if (lane == 31) s_warp[warp] = before;
        bad = __syncthreads_or(bad);
        if (bad) {
            if (tid == 0) set_status(KDA_ERR_BAD_SEQLENS);
            return;
        }
        long long total = 0;
        before -= mine;
        for (int i = 0; i < W; ++i) {
            if (i < warp) before += s_warp[i];
            total += s_warp[i];
        }
        s_before[tid] = before;
        share = max((total + gridDim.x - 1) / gridDim.x, (long long)F4_SHARE);
        const long long begin = share * blockIdx.x, end = min(begin + share, total);
        if (begin >= end) return;
        __syncthreads();
        const long long sub = (share + W - 1) / W, start = begin + sub * warp;
        w.left = min(sub, end - start);
        if (w.left > 0) {
            // the last thread whose requests begin at or before the start (ones of length 0 share their place with the next)
            int at = 0;
            for (int i = lane; i < L::THREADS; i += 32)
                if (s_before[i] <= start) at = i;
            at = __reduce_max_sync(0xffffffffu, at);
            long long x = start - s_before[at], head = 0;
            for (w.n = at * per;; ++w.n) {
                w.r.load(p, w.n, ROWS);
                head = w.r.length(p, ROWS);
                if (x < head * p.a.H_kv) break;
                x -= head * p.a.H_kv;
            }
            w.hk = (int)(x / head);
            x -= w.hk * head;
            w.unit = 0;
            for (int n; x >= (n = w.r.chunks(p, (w.unit + 1) * ROWS) + p.unit_cost); ++w.unit) x -= n;
            w.at = (int)x;
        }
    }

    // ---- loads: STAGES - 1 chunks ahead of the one that is worked on; the block ids are looked up a chunk earlier still
    const uint32_t ring = sbase + warp * L::RING;
    const int box = min(F4_KEYS, 1 << p.a.block_log2);   // rows of a chunk in one block
    F4Walk &ahead = s_ahead[warp];
    int ahead_c = 0, ahead_end = 0, ahead_seen = 0, ahead_hk = 0;
    const int32_t *ahead_table = nullptr;
    bool more;
    auto next_piece = [&](F4Walk &x) {
        more = x.next(p, ROWS);
        __syncwarp();
        if (lane == 0) ahead = x;
        __syncwarp();
        ahead_c = x.a;
        ahead_end = x.b;
        ahead_seen = x.seen;
        ahead_hk = x.hk;
        ahead_table = p.a.table + (size_t)x.n * p.a.max_blocks;
    };
    {
        F4Walk x = w;
        next_piece(x);
    }
    int id[2], id_row = 0, id_hk = 0;   // blocks of the next chunk's halves (-2: nothing to load)
    auto look_up = [&]() {
        const int key = ahead_c * F4_KEYS;
        id[0] = id[1] = -2;
        if (more && key < ahead_seen) {
            const int e = key >> p.a.block_log2;
            id[0] = max(ahead_table[e], -1);
            if (box != F4_KEYS && key + box < ahead_seen) id[1] = max(ahead_table[e + 1], -1);
        }
        id_row = key & ((1 << p.a.block_log2) - 1);
        id_hk = ahead_hk;
        if (more && ++ahead_c == ahead_end) {
            F4Walk x = ahead;
            next_piece(x);
        }
    };
    // 16-byte pieces of codes: a lane's row and place, exchanged so that neither product's reads collide
    constexpr int PER_ROW = ROWB / 16, COPIES = F4_KEYS * PER_ROW / 32;
    const uint32_t copy_row = lane / PER_ROW, copy_at = lane % PER_ROW;
    const uint32_t copy_to = copy_row * ROWB + ((copy_at ^ (D == 128 ? copy_row >> 1 & 3u : copy_row >> 2 & 1u)) << 4);
    const uint32_t slab_bytes = (uint32_t)q4_row_bytes(D) << p.a.block_log2;
    // scales: the first lanes for keys, as many behind them for values
    const int scale_lanes = box * (D / 32) / 16, scale_v = lane >= scale_lanes, scale_x = lane - (scale_v ? scale_lanes : 0);
    const uint32_t scale_to = 2 * L::CODES + scale_v * L::SCALES + 16 * scale_x;
    // (blocks of 16 rows: the lanes behind those, for the second block)
    const int lane2 = lane - 2 * scale_lanes, second_v = lane2 >= scale_lanes, second_x = lane2 - (second_v ? scale_lanes : 0);
    const uint32_t scale_second = 2 * L::CODES + second_v * L::SCALES + 16 * (scale_lanes + second_x);
    const uint8_t *scale_from_second = (second_v ? p.a.v : p.a.k) + ((size_t)ROWB << p.a.block_log2) + 16 * second_x;
    const uint8_t *k_from = p.a.k + 16 * lane, *v_from = p.a.v + 16 * lane;
    const uint8_t *scale_from = (scale_v ? p.a.v : p.a.k) + ((size_t)ROWB << p.a.block_log2) + 16 * scale_x;
    auto load = [&](uint32_t to) {   // the chunk that look_up found, into the stage at `to`
        const uint32_t blocks = p.a.num_blocks;
        if (box == F4_KEYS && (uint32_t)id[0] < blocks) {
            const size_t slab = (size_t)((uint32_t)id[0] * (uint32_t)p.a.H_kv + (uint32_t)id_hk) * slab_bytes;
            const uint8_t *k = k_from + slab + id_row * ROWB, *v = v_from + slab + id_row * ROWB;
            const uint32_t at = to + copy_to;
            cp16_at<0, 0>(at, k);
            cp16_at<512, 512>(at, k);
            cp16_at<L::CODES, 0>(at, v);
            cp16_at<L::CODES + 512, 512>(at, v);
            if constexpr (COPIES == 4) {
                cp16_at<1024, 1024>(at, k);
                cp16_at<1536, 1536>(at, k);
                cp16_at<L::CODES + 1024, 1024>(at, v);
                cp16_at<L::CODES + 1536, 1536>(at, v);
            }
            if (lane < 2 * scale_lanes) cp_async16(to + scale_to, scale_from + slab + id_row * (D / 32));
        } else if (box != F4_KEYS && (uint32_t)id[0] < blocks && (uint32_t)id[1] < blocks) {
            // two blocks of 16 rows (124 against 151 us in the loop below, 256 decoded tokens over 2040 keys; 118 with larger blocks)
            const size_t slab = (size_t)((uint32_t)id[0] * (uint32_t)p.a.H_kv + (uint32_t)id_hk) * slab_bytes;
            const size_t next = (size_t)((uint32_t)id[1] * (uint32_t)p.a.H_kv + (uint32_t)id_hk) * slab_bytes;
            const uint8_t *k = k_from + slab, *v = v_from + slab, *k1 = k_from + next, *v1 = v_from + next;
            const uint32_t at = to + copy_to;
            cp16_at<0, 0>(at, k);
            cp16_at<L::CODES, 0>(at, v);
            cp16_at<16 * ROWB, 0>(at, k1);
            cp16_at<L::CODES + 16 * ROWB, 0>(at, v1);
            if constexpr (COPIES == 4) {
                cp16_at<512, 512>(at, k);
                cp16_at<L::CODES + 512, 512>(at, v);
                cp16_at<16 * ROWB + 512, 512>(at, k1);
                cp16_at<L::CODES + 16 * ROWB + 512, 512>(at, v1);
            }
            // (twice the lanes for the scales, each of its block's)
            const bool second = lane >= 2 * scale_lanes;
            if (lane < 4 * scale_lanes)
                cp_async16(to + (second ? scale_second : scale_to), (second ? scale_from_second + next : scale_from + slab));
        } else {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int b = h ? id[1] : id[0];
                if (b == -2) continue;
                const bool good = (uint32_t)b < (uint32_t)p.a.num_blocks;
                if (!good) set_status(KDA_ERR_BAD_PAGES);
                const size_t slab = (size_t)((uint32_t)(good ? b : 0) * (uint32_t)p.a.H_kv + (uint32_t)id_hk) * slab_bytes;
                const uint8_t *k = k_from + slab + id_row * ROWB, *v = v_from + slab + id_row * ROWB;
                const uint32_t at = to + copy_to + h * box * ROWB, scales = to + scale_to + h * box * (D / 32);
                const float zeros = __uint_as_float(0x88888888u);   // codes of zeros, for rows without a block
                for (int i = 0; i < box * PER_ROW / 32; ++i) {
                    if (good) {
                        cp_async16(at + 512 * i, k + 512 * i);
                        cp_async16(at + 512 * i + L::CODES, v + 512 * i);
                    } else {
                        sts_f4(at + 512 * i, make_float4(zeros, zeros, zeros, zeros));
                        sts_f4(at + 512 * i + L::CODES, make_float4(zeros, zeros, zeros, zeros));
                    }
                }
                if (lane < 2 * scale_lanes) {
                    if (good) cp_async16(scales, scale_from + slab + id_row * (D / 32));
                    else sts_f4(scales, make_float4(0.f, 0.f, 0.f, 0.f));
                }
            }
        }
        cp_async_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        load(ring + i * L::STAGE);
        look_up();
    }
    uint32_t to = (S - 1) * L::STAGE, at = 0;   // places in the ring of the next chunk to load, to work on
    auto advance = [](uint32_t &place) { place = place == L::RING - L::STAGE ? 0 : place + L::STAGE; };

    // ---- attention
    {
        const int g = lane >> 2, t = lane & 3, odd = t & 1;
        // Keys of score rows g and g + 8 are kr and kr + 8: neighbours change places where g / 2 is odd, so that the lanes
        // of a value's read, two rows apart, find different banks.
        const int kr = (g & ~1) + ((g & 1) ^ ((g >> 1) & 1));
        // shared-memory offsets in a chunk (swizzled: 16-byte pieces of a row are exchanged by the row's place)
        uint32_t k_at[BLOCKS], v_at[2];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) k_at[b] = kr * ROWB + 4 * t + ((b ^ (D == 128 ? kr >> 1 & 3 : kr >> 2 & 1)) << 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * t + (i ^ odd);
            v_at[i] = L::CODES + r * ROWB +
                      (D == 128 ? (((g >> 1) ^ (r >> 1 & 3)) << 4) + 8 * (g & 1) : (((g >> 2) ^ (r >> 2 & 1)) << 4) + 4 * (g & 3));
        }
        // Pair j of a word as fp16, below the normal numbers: 2^-24 c where the code is in bits 0 .. 3 of each half (j = 0,
        // and j = 2 8 bits further down), 2^-20 c where it is in bits 4 .. 7 (j = 1, 3)
        auto codes_f16 = [](uint32_t word, int j) { return (j < 2 ? word : word >> 8) & (j & 1 ? 0x00f000f0u : 0x000f000fu); };
        // which scale bytes of two keys' words make a pair
        const uint32_t blk = D == 128 ? g >> 1 : g >> 2, second = D == 128 ? 4 + blk : 2 + blk;
        const uint32_t sel = odd ? second | blk << 8 : blk | second << 8;

        while (w.next(p, ROWS)) {
            {
                // ---- queries: columns g of the products, as fp16 with the row's largest magnitude between 2^14 and 2^15, so
                // that a channel is itself down to 2^-27 of that.  A lane's channels are those of its words of a key, 8 in
                // each block of 32.  Codes come as 2^-24 c and 2^-20 c = 2^-24 (c 2^4), whose queries are 2^-4 of the others,
                // and c is 8 + n: a block's product is off by 2^-24 8 times the queries' sum.
                uint32_t q[TILES][BLOCKS][4];
                float2 excess[TILES][BLOCKS], m[TILES], minus_m[TILES], l[TILES], factor[TILES];
                int limit[TILES][2];
                float o[MT][TILES][4];
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
                    const bool real = 8 * n + g < w.rows;
                    const uint16_t *src = p.a.q + out_row(p, w.r, w.hk, w.first + 8 * n + g) * D;
                    uint32_t most = 0;
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) {
                        const uint4 u = real ? *reinterpret_cast<const uint4 *>(src + 32 * b + 8 * t) : make_uint4(0, 0, 0, 0);
                        q[n][b][0] = u.x; q[n][b][1] = u.y; q[n][b][2] = u.z; q[n][b][3] = u.w;
#pragma unroll
                        for (int j = 0; j < 4; ++j) most = max(most, max(q[n][b][j] << 16 & 0x7fff0000u, q[n][b][j] & 0x7fff0000u));
                    }
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    // up and down are reciprocal powers of two; exponent fields from 14 to 253
                    const uint32_t e = most ? min(268u - (most >> 23), 253u) : 127u;
                    const float up = __uint_as_float(e << 23);
                    const float down = most >= 0x7f800000u ? NAN : __uint_as_float((254u - e) << 23);
                    // queries 2t and 2t + 1 are the columns of this lane's scores.  (A factor past the range would make a score of
                    // 0 NaN; under one at the range's end any other is still too far away to share the weight.)
                    const float mine = p.c * down, f = fabsf(mine) == INFINITY ? copysignf(FLT_MAX, mine) : mine;
                    factor[n] = make_float2(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) {
                        float sum = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x0 = bf16_lo(q[n][b][j]) * up, x1 = bf16_hi(q[n][b][j]) * up;
                            q[n][b][j] = j & 1 ? pack_f16x2(x0 * 0x1p-4f, x1 * 0x1p-4f) : pack_f16x2(x0, x1);
                            sum = fmaf(-0x1p-21f, x0 + x1, sum);
                        }
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                        excess[n][b] = make_float2(__shfl_sync(0xffffffffu, sum, 8 * t), __shfl_sync(0xffffffffu, sum, 8 * t + 4));
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        limit[n][x] = w.r.keys - w.r.fresh + f4_token(p, min(w.first + 8 * n + 2 * t + x, w.first + w.rows - 1)) + 1;
                    // -m, finite: without a reference yet, scores of -infinity weigh nothing and any other makes a chunk look
                    m[n] = make_float2(-INFINITY, -INFINITY);
                    minus_m[n] = make_float2(FLT_MAX, FLT_MAX);
                    l[n] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int i = 0; i < MT; ++i) o[i][n][x] = 0.f;
                }
                const int lowest = w.r.keys - w.r.fresh + f4_token(p, w.first) + 1;   // of the rows' limits

                for (int c = w.a; c < w.b; ++c) {
                    load(ring + to);
                    advance(to);
                    look_up();
                    cp_async_wait<S - 1>();
                    __syncwarp();
                    // plain loads, whose offsets go into the instructions
                    const unsigned char *stage = sm + warp * L::RING + at;
                    advance(at);
                    const unsigned char *k_scales = stage + 2 * L::CODES + (D == 128 ? kr : kr & ~1) * (D / 32);
                    const unsigned char *v_scales = stage + 2 * L::CODES + L::SCALES + 2 * t * (D / 32);
                    auto word = [](const unsigned char *at) { return *reinterpret_cast<const uint32_t *>(at); };
                    auto pair = [](const unsigned char *at) { return *reinterpret_cast<const uint2 *>(at); };
                    // ---- scores: sum over blocks of 32 channels of the keys' scale times the codes' product with q
                    float2 s[TILES][4];   // of keys 16 (i / 2) + 8 (i % 2) + kr
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t w0, w1;   // scale bytes of two keys
                        if (D == 128) {
                            w0 = word(k_scales + 16 * mt * 4);
                            w1 = word(k_scales + (16 * mt + 8) * 4);
                        } else {
                            w0 = word(k_scales + 16 * mt * 2) >> (16 * (kr & 1));
                            w1 = word(k_scales + (16 * mt + 8) * 2) >> (16 * (kr & 1));
                        }
#pragma unroll
                        for (int b = 0; b < BLOCKS; ++b) {
                            const uint32_t x0 = word(stage + k_at[b] + 16 * mt * ROWB), x1 = word(stage + k_at[b] + (16 * mt + 8) * ROWB);
                            // the scales times 2^24
                            const float s0 = __uint_as_float(__byte_perm(w0, 0, 0x4440 | b) * p.two20 + 0x44000000u);
                            const float s1 = __uint_as_float(__byte_perm(w1, 0, 0x4440 | b) * p.two20 + 0x44000000u);
                            uint32_t a[8];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                a[2 * j] = codes_f16(x0, j);
                                a[2 * j + 1] = codes_f16(x1, j);
                            }
#pragma unroll
                            for (int n = 0; n < TILES; ++n) {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(d, a[0], a[1], a[2], a[3], q[n][b][0], q[n][b][1]);
                                mma_f16(d, a[4], a[5], a[6], a[7], q[n][b][2], q[n][b][3]);
                                const float2 d0 = __fadd2_rn(make_float2(d[0], d[1]), excess[n][b]);
                                const float2 d1 = __fadd2_rn(make_float2(d[2], d[3]), excess[n][b]);
                                s[n][2 * mt] = b ? __ffma2_rn(make_float2(s0, s0), d0, s[n][2 * mt]) : __fmul2_rn(make_float2(s0, s0), d0);
                                s[n][2 * mt + 1] = b ? __ffma2_rn(make_float2(s1, s1), d1, s[n][2 * mt + 1]) : __fmul2_rn(make_float2(s1, s1), d1);
                            }
                        }
                    }
                    // ---- weights
                    const bool edge = (c + 1) * F4_KEYS > lowest;
                    float2 fac[TILES];
#pragma unroll
                    for (int n = 0; n < TILES; ++n) fac[n] = factor[n];
                    if (edge) {   // keys that a row does not see; scores in units of log 2 from here on
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int key = c * F4_KEYS + 16 * (i >> 1) + kr + 8 * (i & 1);
                                s[n][i].x = key >= limit[n][0] ? -INFINITY : s[n][i].x * factor[n].x;
                                s[n][i].y = key >= limit[n][1] ? -INFINITY : s[n][i].y * factor[n].y;
                            }
                            fac[n] = make_float2(1.f, 1.f);
                        }
                    }
                    uint32_t pk[TILES][4];
                    float2 sum[TILES];
                    auto weights = [&]() {
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            sum[n] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float2 y = __ffma2_rn(s[n][i], fac[n], minus_m[n]);
                                y.x = ex2(y.x);
                                y.y = ex2(y.y);
                                sum[n] = __fadd2_rn(sum[n], y);
                                pk[n][i] = pack_bf16x2(y.x, y.y);
                            }
                        }
                    };
                    // A row that sees no key of the piece's first chunk sees none of the piece: its reference stays -infinity.  (It also
                    // does where all that it sees scores below the lowest number, until another score makes a chunk look.)
                    bool look = c == w.a;
                    if (!look) {
                        weights();
                        float most = sum[0].x + sum[0].y;
#pragma unroll
                        for (int n = 1; n < TILES; ++n) most += sum[n].x + sum[n].y;
                        look = __any_sync(0xffffffffu, !(most <= F4_MOST));
                    }
                    if (look) {
                        bool move = false;
                        float2 f[TILES];
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            auto raise = [&](float top, float &m, float &minus_m, float &l) {   // returns what is there's factor
#pragma unroll
                                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                                if (!(top > m + 8.f)) return 1.f;
                                const float f = ex2(m - top);
                                m = top;
                                minus_m = -fminf(top, FLT_MAX);   // (a score above the range weighs infinitely: NaN in the end)
                                l *= f;
                                move = true;
                                return f;
                            };
                            float2 top = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                top.x = fmaxf(top.x, s[n][i].x * fac[n].x);
                                top.y = fmaxf(top.y, s[n][i].y * fac[n].y);
                            }
                            f[n].x = raise(top.x - Q4_LOG_UP, m[n].x, minus_m[n].x, l[n].x);
                            f[n].y = raise(top.y - Q4_LOG_UP, m[n].y, minus_m[n].y, l[n].y);
                        }
                        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                            for (int n = 0; n < TILES; ++n)
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const float fx = x & 1 ? f[n].y : f[n].x;
#pragma unroll
                                    for (int i = 0; i < MT; ++i) o[i][n][x] *= fx;
                                }
                        }
                        weights();
                    }
#pragma unroll
                    for (int n = 0; n < TILES; ++n) l[n] = __fadd2_rn(l[n], sum[n]);
                    // ---- outputs
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t bq[TILES][2];
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            bq[n][0] = transpose_8x8(pk[n][2 * mt]);
                            bq[n][1] = transpose_8x8(pk[n][2 * mt + 1]);
                        }
                        Q4Scale scale[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t x;
                            if (D == 128) {
                                const uint2 y = pair(v_scales + (16 * mt + 8 * i) * 4);
                                x = __byte_perm(y.x, y.y, sel) & 0x00ff00ffu;
                            } else {
                                x = __byte_perm(word(v_scales + (16 * mt + 8 * i) * 2), 0, sel) & 0x00ff00ffu;
                            }
                            scale[i] = q4_scales(x, p.two4);
                        }
                        uint32_t v[4][D / 64];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (D == 128) {
                                const uint2 x = pair(stage + v_at[i & 1] + (16 * mt + 8 * (i >> 1)) * ROWB);
                                v[i][0] = x.x;
                                v[i][D / 64 - 1] = x.y;
                            } else {
                                v[i][0] = word(stage + v_at[i & 1] + (16 * mt + 8 * (i >> 1)) * ROWB);
                            }
                        }
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            const uint32_t lo01 = __byte_perm(v[0][x], v[1][x], 0x5410), hi01 = __byte_perm(v[0][x], v[1][x], 0x7632);
                            const uint32_t lo23 = __byte_perm(v[2][x], v[3][x], 0x5410), hi23 = __byte_perm(v[2][x], v[3][x], 0x7632);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t a0 = q4_pair(lo01, j, scale[0]), a1 = q4_pair(hi01, j, scale[0]);
                                const uint32_t a2 = q4_pair(lo23, j, scale[1]), a3 = q4_pair(hi23, j, scale[1]);
#pragma unroll
                                for (int n = 0; n < TILES; ++n) mma_bf16(o[4 * x + j][n], a0, a1, a2, a3, bq[n][0], bq[n][1]);
                            }
                        }
                    }
                    __syncwarp();   // the stage is free
                }
                // ---- the piece's rows: a whole unit's go out, a part of one stays for its joining
                const bool whole = w.a == 0 && w.b == w.all;
                const uint32_t part = w.a > 0 ? 0 : 1;
                const uint32_t part_at = part ? ring : sbase + L::PART + warp * L::PART_WARP;
                if (!whole && part) cp_async_wait<0>();   // (nothing is in flight in the ring any more)
#pragma unroll
                for (int n = 0; n < TILES; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {   // queries 2t and 2t + 1
                        float sum = x ? l[n].y : l[n].x;
                        const float ref = x ? m[n].y : m[n].x;
#pragma unroll
                        for (int lanes = 4; lanes < 32; lanes <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, lanes);
                        const int row = 8 * n + 2 * t + x;
                        float y[D / 8];   // channels (D / 8) g ..
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            y[2 * i] = o[i][n][x] * Q4_UP;
                            y[2 * i + 1] = o[i][n][2 + x] * Q4_UP;
                        }
                        if (!whole) {
                            if (g == 0) sts_f2(sbase + L::ML + ((warp * 2 + part) * ROWS + row) * 8, make_float2(ref, sum));
                            const uint32_t at = part_at + row * L::PART_ROW;
#pragma unroll
                            for (int i = 0; i < D / 32; ++i)
                                sts_f4(at + (((D / 32) * g + i) ^ t) * 16, make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
                        } else if (row < w.rows) {
                            const size_t at = out_row(p, w.r, w.hk, w.first + row);
                            if (limit[n][x] <= 0) sum = 0.f;   // no key, under a NaN scale too
                            const bool none = sum == 0.f;
                            const float inv = none ? 0.f : 1.f / sum;
                            uint32_t u[D / 16];
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) u[i] = none ? 0 : pack_bf16x2(y[2 * i] * inv, y[2 * i + 1] * inv);
#pragma unroll
                            for (int i = 0; i < D / 64; ++i)
                                *reinterpret_cast<uint4 *>(p.a.out + at * D + (D / 8) * g + 8 * i) =
                                    make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                            if (g == 0 && p.a.lse) p.a.lse[at] = none ? -INFINITY : (ref + lg2(sum)) * (1.f / LOG2E);
                        }
                    }
                if (!whole && lane == 0) s_part[warp][part] = F4Part{w.n, w.hk, w.first, w.rows, true, w.b == w.all, w.rest};
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- joining what the shares' ends cut: a unit's parts lie in neighbouring warps, the first of them the part that
    // a warp ends with, or the first warp's that it begins with (the unit's beginning is another CTA's then)
    for (int i = -1; i < W; ++i) {
        if (!s_part[max(i, 0)][i < 0 ? 0 : 1].there) continue;
        const F4Part d = s_part[max(i, 0)][i < 0 ? 0 : 1];
        int last = max(i, 0);
        bool ends = d.ends;
        long long rest = d.rest;
        while (!ends && last + 1 < W && s_part[last + 1][0].there) {
            ++last;
            ends = s_part[last][0].ends;
            rest = s_part[last][0].rest;
        }
        const bool closed = i >= 0 && ends;
        if (!closed && i >= 0 && tid == 0)
            p.join[blockIdx.x] = F4Join{d.n, d.hk, d.first, d.rows, 1 + (int)((rest + share - 1) / share)};
        constexpr int PIECES = D / 4;
        for (int row = (warp + i + W) % W; row < d.rows; row += W) {
            if (lane >= PIECES) continue;
            auto ml_of = [&](int k) { return lds_f2(sbase + L::ML + ((k * 2 + (k == i ? 1 : 0)) * ROWS + row) * 8); };
            float top = -INFINITY, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = max(i, 0); k <= last; ++k) top = fmaxf(top, ml_of(k).x);
            const float ref = top == -INFINITY ? 0.f : top;
            for (int k = max(i, 0); k <= last; ++k) {
                const float2 ml = ml_of(k);
                const uint32_t at = k == i ? sbase + k * L::RING : sbase + L::PART + k * L::PART_WARP;
                const float4 x = lds_f4(at + row * L::PART_ROW + ((lane ^ (row >> 1 & 3)) << 4));
                const float f = ex2(ml.x - ref);
                sum += f * ml.y;
                acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
            }
            if (closed) {
                F4Request r;
                r.load(p, d.n, ROWS);
                const size_t at = out_row(p, r, d.hk, d.first + row);
                if (r.seen(p, d.first + row + 1) <= 0) sum = 0.f;   // no key, under a NaN scale too
                const bool none = sum == 0.f;
                const float inv = none ? 0.f : 1.f / sum;
                *reinterpret_cast<uint2 *>(p.a.out + at * D + 4 * lane) =
                    none ? make_uint2(0, 0) : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                if (lane == 0 && p.a.lse) p.a.lse[at] = none ? -INFINITY : (ref + lg2(sum)) * (1.f / LOG2E);
            } else {
                const int slot = 2 * blockIdx.x + (i < 0 ? 0 : 1);
                *reinterpret_cast<float4 *>(p.o + ((size_t)slot * F4_MAX_ROWS + row) * D + 4 * lane) = acc;
                if (lane == 0) p.ml[slot * F4_MAX_ROWS + row] = make_float2(sum == 0.f ? -INFINITY : top, sum);
            }
        }
    }
}

template <int D>
__global__ __launch_bounds__(256) void attn_q4_join_kernel(const F4Params p) {
    grid_dep_wait();   // launched while the pieces are still being computed
    f4_join<D>(p, blockIdx.x, blockIdx.y * 256 + threadIdx.x);
}

// ---------------------------------------------------------------- host side
namespace {
template <int D, int ROWS>
cudaError_t run(const F4Params &p, int grid, cudaStream_t stream) {
    using L = F4Layout<D, ROWS>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static bool ready[64] = {false};   // by device: the attribute is set once
    if (!ready[dev & 63]) {
        e = cudaFuncSetAttribute(attn_q4_few_kernel<D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::BYTES);
        if (e != cudaSuccess) return e;
        ready[dev & 63] = true;
    }
    attn_q4_few_kernel<D, ROWS><<<grid, L::THREADS, L::BYTES, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t join(const F4Params &p, int rows, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, (rows * (D / 4) + 255) / 256);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_q4_join_kernel<D>, p);
}
}  // namespace

// Rows a unit has, 8 or 16: those that a request has on average, or a single token's where the average is the other
// kernel's.  A key's codes are expanded once a unit, but tiles of 16 columns leave registers for fewer warps.  128
// requests over 4096 keys, 8 and 16: with 8 rows over 4 heads 67 and 94 us, with 9 116 and 94, with 12 over 8 heads 215
// and 172, with 32 412 and 325.
int attn_q4_few_rows(const AttnQ4Args &a, int most_rows) {
    const int G = a.H_q / a.H_kv;
    const long long rows = ((long long)a.T + a.N - 1) / a.N * G;
    return (rows > most_rows ? G : rows) <= 8 ? 8 : 16;
}

F4Params attn_q4_few_params(const AttnQ4Args &a, int most_rows, void *ws) {
    F4Params p;
    p.a = a;
    char *base = static_cast<char *>(ws);
    p.join = reinterpret_cast<F4Join *>(base);
    base += align256(sizeof(F4Join) * MAX_SMS);
    p.ml = reinterpret_cast<float2 *>(base);
    base += align256(sizeof(float2) * 2 * MAX_SMS * F4_MAX_ROWS);
    p.o = reinterpret_cast<float *>(base);
    p.c = a.scale * LOG2E;
    p.G = a.H_q / a.H_kv;
    p.over_g = (65536u + p.G - 1) / p.G;
    p.most_rows = most_rows;
    // About 4000 cycles of a warp, whose chunks take 2700.  0, 2 and 4: 256 decoded tokens over 300 keys 34.2, 32.6 and 32.3
    // us, 64 over 4096 65.7, 66.2 and 67.5; 128 x 16 rows over 1024 60.7, 60.5 and 61.3
    p.unit_cost = 2;
    p.two20 = 1u << 20;
    p.two4 = 1u << 4;
    return p;
}

size_t attn_q4_few_workspace_bytes(int D) {
    return align256(sizeof(F4Join) * MAX_SMS) + align256(sizeof(float2) * 2 * MAX_SMS * F4_MAX_ROWS) +
           sizeof(float) * 2 * MAX_SMS * F4_MAX_ROWS * D;
}

cudaError_t launch_attn_q4_few(const F4Params &p, int rows, cudaStream_t stream, int *launches) {
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    ++*launches;
    if (rows == 8) return p.a.D == 64 ? run<64, 8>(p, sms, stream) : run<128, 8>(p, sms, stream);
    return p.a.D == 64 ? run<64, 16>(p, sms, stream) : run<128, 16>(p, sms, stream);
}

cudaError_t launch_attn_q4_few_join(const F4Params &p, int rows, cudaStream_t stream, int *launches) {
    const int sms = sm_count();
    ++*launches;
    return p.a.D == 64 ? join<64>(p, rows, sms, stream) : join<128>(p, rows, sms, stream);
}

}  // namespace kda
