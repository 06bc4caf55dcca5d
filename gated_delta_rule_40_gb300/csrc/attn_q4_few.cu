// Attention of few query rows over the 4-bit cache (see attn_q4.cu for which requests these are).
#include "attn_q4_few.cuh"

namespace kda {
namespace {

__device__ __forceinline__ bool f4_try(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
    return done != 0;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a));
    return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 x;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a));
    return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
    return x;
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
__device__ __forceinline__ void sts_f2(uint32_t a, float2 x) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x.x), "f"(x.y) : "memory");
}

template <int D, int ROWS>
__global__ __launch_bounds__(F4Layout<D, ROWS>::THREADS, 1) void attn_q4_few_kernel(const __grid_constant__ CUtensorMap tk,
                                                                                     const __grid_constant__ CUtensorMap tv,
                                                                                     const __grid_constant__ F4Params p) {
    using L = F4Layout<D, ROWS>;
    constexpr int W = L::WARPS, S = L::STAGES, TILES = L::TILES, QT = L::QT, MT = D / 16, BLOCKS = D / 32, ROWB = D / 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = aligned_smem<1024>(smem_raw);
    const uint32_t sbase = smem_u32(sm), bar = sbase + L::BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::FLAG);
    __shared__ long long s_warp[W + 1], s_x;
    __shared__ int s_n;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    grid_dep_launch();

    // ---- this CTA's share of the line of all units
    F4Walk w;
    {
        bool bad = false;
        if (tid == 0) {
            p.join[blockIdx.x].pieces = 0;
            bad = p.a.cu[0] != 0 || p.a.cu[p.a.N] > p.a.T;
            for (int i = 0; i < L::COUNT; ++i) mbar_init(bar + 8 * i, i >= L::PF && i < L::PE ? W : 1);
            mbar_fence_init();
            *abort_flag = 0;
        }
        const long long most = min((long long)p.a.max_blocks << p.a.block_log2, F4_MAX_KEYS);
        const int per = (p.a.N + L::THREADS - 1) / L::THREADS, n0 = min(tid * per, p.a.N), n1 = min(n0 + per, p.a.N);
        long long mine = 0;
        F4Request r;
        for (int n = n0; n < n1; ++n) {
            r.load(p, n, ROWS);
            if (r.fresh < 0 || r.keys < 0 || r.keys > most) bad = true;
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
        for (int i = 0; i <= W; ++i) {
            if (i < warp) before += s_warp[i];
            total += s_warp[i];
        }
        const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)F4_SHARE);
        const long long start = share * blockIdx.x;
        w.left = min(share, total - start);
        if (w.left <= 0) return;
        if (start >= before && start < before + mine) {
            long long x = start - before;
            for (int n = n0;; ++n) {
                r.load(p, n, ROWS);
                const long long len = r.length(p, ROWS) * p.a.H_kv;
                if (x < len) {
                    s_n = n;
                    s_x = x;
                    break;
                }
                x -= len;
            }
        }
        __syncthreads();
        w.n = s_n;
        w.r.load(p, w.n, ROWS);
        const long long head = w.r.length(p, ROWS);
        w.hk = (int)(s_x / head);
        long long x = s_x - w.hk * head;
        w.unit = 0;
        for (int n; x >= (n = w.r.chunks(p, (w.unit + 1) * ROWS) + p.unit_cost); ++w.unit) x -= n;
        w.at = (int)x;
    }
    const long long share = w.left;   // a full share wherever a unit is cut by its end

    bool ok = true;
    constexpr uint32_t LIMIT = 1u << 22;
    auto wait = [&](int b, uint32_t parity) {   // by each lane for itself
        if (f4_try(bar + 8 * b, parity)) return true;
        for (uint32_t i = 0; i < LIMIT; ++i) {
            if (f4_try(bar + 8 * b, parity)) return true;
            if ((i & 63) == 63 && *abort_flag) break;
        }
        return ok = false;
    };
    uint32_t run = 0;   // chunks of the share's earlier pieces: chunk i goes to warp i % W

    if (warp == W) {
        // ------------------------------------------------------------ loader: four chunks at a time, a lane a copy
        const int sub = lane >> 3, op = lane & 7, kv = op & 1, scales = (op >> 1) & 1, half = op >> 2;
        const int box = min(F4_KEYS, 1 << p.a.block_log2), halves = F4_KEYS / box;
        const CUtensorMap *map = kv ? &tv : &tk;
        const uint8_t *cache = kv ? p.a.v : p.a.k;
        while (__all_sync(0xffffffffu, ok) && w.next(p, ROWS)) {
            // block of this lane's rows of chunk c: -1 one outside the cache, -2 nothing to load
            auto page = [&](int c) {
                const int key = c * F4_KEYS + half * box;
                if (c >= w.b || half >= halves || key >= w.seen) return -2;
                const int id = p.a.table[(size_t)w.n * p.a.max_blocks + (key >> p.a.block_log2)];
                return id >= 0 && id < p.a.num_blocks ? id : -1;
            };
            int id = page(w.a + sub);
            for (int c0 = w.a; c0 < w.b; c0 += 4) {
                const int next_id = page(c0 + 4 + sub), c = c0 + sub;
                const bool active = c < w.b;
                const uint32_t i = run + (uint32_t)(c - w.a), k = i / W, slot = (i - k * W) * S + k % S, use = k / S;
                if (active && use > 0) wait(L::EMPTY + slot, (use - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                const uint32_t have = __ballot_sync(0xffffffffu, id >= 0) >> (8 * sub) & 0xffu;
                const uint32_t missing = __ballot_sync(0xffffffffu, id == -1) >> (8 * sub) & 0xffu;
                const uint32_t full = bar + 8 * (L::FULL + slot);
                if (active && op == 0) {
                    if (missing) set_status(KDA_ERR_BAD_PAGES);
                    *reinterpret_cast<volatile uint32_t *>(sm + L::BADS + 4 * slot) = (missing & 1u) | (missing >> 3 & 2u);
                    mbar_expect_tx(full, (uint32_t)(((have & 1u) + (have >> 4 & 1u)) * box * 2 * (ROWB + D / 32)));
                }
                __syncwarp();
                if (id >= 0) {
                    const int row = (c * F4_KEYS + half * box) & ((1 << p.a.block_log2) - 1);
                    const long long slab = (long long)id * p.a.H_kv + w.hk;
                    if (scales) {
                        const uint32_t dst = sbase + L::SC + slot * L::SC_STAGE + kv * L::SCALES + half * box * (D / 32);
                        bulk_g2s(dst, cache + (((size_t)slab * q4_row_bytes(D) + ROWB) << p.a.block_log2) + row * (D / 32),
                                 (uint32_t)box * (D / 32), full);
                    } else {
                        tma_load_3d(sbase + slot * L::STAGE + kv * L::CODES + half * box * ROWB, map, 0, row, (int)slab, full);
                    }
                }
                id = next_id;
            }
            run += (uint32_t)(w.b - w.a);
        }
    } else {
        // ------------------------------------------------------------ attention
        const int g = lane >> 2, t = lane & 3, odd = t & 1;
        const int kr = 4 * (g >> 1) + ((g & 1) ^ ((g >> 1) & 1));   // key of score row g; row g + 8's is kr + 2
        // shared-memory offsets in a chunk (swizzled: 16-byte pieces of a row are exchanged by the row's place)
        const uint32_t k_at = kr * ROWB + 4 * t, k_x0 = D == 128 ? (kr >> 1 & 3) << 4 : (kr >> 2 & 1) << 4;
        const uint32_t k_x1 = D == 128 ? ((kr + 2) >> 1 & 3) << 4 : k_x0;   // (D = 64: 4 rows share a pattern)
        uint32_t v_at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * t + (i ^ odd);
            v_at[i] = L::CODES + r * ROWB +
                      (D == 128 ? (((g >> 1) ^ (r >> 1 & 3)) << 4) + 8 * (g & 1) : (((g >> 2) ^ (r >> 2 & 1)) << 4) + 4 * (g & 3));
        }
        // which scale bytes of two keys' words make a pair
        const uint32_t blk = D == 128 ? g >> 1 : g >> 2, second = D == 128 ? 4 + blk : 2 + blk;
        const uint32_t sel = odd ? second | blk << 8 : blk | second << 8;

        uint32_t k_use = 0, pieces = 0;   // chunks and pieces of this warp so far
        while (ok && w.next(p, ROWS)) {
            const int n_chunks = w.b - w.a, parts = min(W, n_chunks);
            const int shift = (int)((warp + W - run % W) % W);
            const uint32_t buf = pieces % L::BUFS, use = pieces / L::BUFS;
            const bool part = shift < n_chunks;
            uint32_t q[TILES][BLOCKS][2];
            float init[TILES][BLOCKS], cq[TILES], m[TILES], l[TILES];
            int limit[TILES];
            float o[MT][QT][4], z[QT][4];
            if (part) {
                // ---- queries: high and low e4m3 halves, with the row's largest magnitude between 128 and 256
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
                    const int qr = 4 * n + (g >> 1);
                    uint4 u[BLOCKS];
                    const bool real = qr < w.rows;
                    const int flat = w.first + qr, tok = flat / p.G;
                    const uint16_t *src = p.a.q + ((size_t)(w.r.row0 + tok) * p.a.H_q + w.hk * p.G + (flat - tok * p.G)) * D;
                    uint32_t most = 0;
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) {
                        u[b] = real ? *reinterpret_cast<const uint4 *>(src + 32 * b + 8 * t) : make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) most = max(most, max(x[j] << 16 & 0x7fff0000u, x[j] & 0x7fff0000u));
                    }
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                    const int e = most ? min(261 - (int)(most >> 23), 253) : 127;   // 6 or more
                    const float up = __uint_as_float((uint32_t)e << 23);
                    const float mine = most >= 0x7f800000u ? NAN : p.c * 512.f * __uint_as_float((uint32_t)(254 - e) << 23);
                    cq[n] = __shfl_sync(0xffffffffu, mine, 8 * t);
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) {
                        const uint32_t x[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
                        float f[8], sum = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            f[2 * j] = bf16_lo(x[j]) * up;
                            f[2 * j + 1] = bf16_hi(x[j]) * up;
                        }
                        // a word's codes come as bytes of channels 0, 4, 1, 5 and 2, 6, 3, 7
                        constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float x0 = f[order[2 * h]], x1 = f[order[2 * h + 1]];
                            uint32_t y = e4m3x2(x0, x1);
                            float2 back = e4m3x2_to_f(y);
                            if (g & 1) {
                                y = e4m3x2(x0 - back.x, x1 - back.y);
                                back = e4m3x2_to_f(y);
                            }
                            sum += back.x + back.y;
                            if ((h & 1) == 0) q[n][b][h >> 1] = y;
                            else q[n][b][h >> 1] |= y << 16;
                        }
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                        init[n][b] = __shfl_sync(0xffffffffu, sum, 8 * t) * (-8.f / 512.f);
                    }
                    limit[n] = w.r.keys - w.r.fresh + min(w.first + 4 * n + t, w.first + w.rows - 1) / p.G + 1;
                    m[n] = -INFINITY;
                    l[n] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < QT; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        z[j][x] = 0.f;
#pragma unroll
                        for (int i = 0; i < MT; ++i) o[i][j][x] = 0.f;
                    }
                const int lowest = w.r.keys - w.r.fresh + w.first / p.G + 1;   // of the rows' limits

                for (int c = w.a + shift; c < w.b; c += W, ++k_use) {
                    const uint32_t stage = k_use % S, slot = warp * S + stage;
                    if (!__all_sync(0xffffffffu, wait(L::FULL + slot, (k_use / S) & 1))) break;
                    const uint32_t codes = sbase + slot * L::STAGE, sc = sbase + L::SC + slot * L::SC_STAGE;
                    const uint32_t lost = *reinterpret_cast<volatile uint32_t *>(sm + L::BADS + 4 * slot);
                    if (lost) {   // rows without a block: codes of zeros, under the smallest scale
                        const int box = min(F4_KEYS, 1 << p.a.block_log2);
                        const float zeros = __uint_as_float(0x88888888u);
                        for (int i = lane; i < 2 * F4_KEYS * (ROWB / 16); i += 32)
                            if (lost >> (i / (ROWB / 16) % F4_KEYS / box) & 1u)
                                sts_f4(codes + 16 * i, make_float4(zeros, zeros, zeros, zeros));
                        for (int i = lane; i < 2 * F4_KEYS; i += 32)
                            if (lost >> (i % F4_KEYS / box) & 1u)
                                for (int b = 0; b < D / 32; ++b) sm[sc - sbase + i * (D / 32) + b] = 0;
                        fence_async_smem();
                        __syncwarp();
                    }
                    // ---- scores: sum over blocks of 32 channels of the keys' scale times the codes' product with q
                    float s[TILES][4];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t w0, w1;   // scale bytes of two keys
                        if (D == 128) {
                            w0 = lds32(sc + (16 * mt + kr) * 4);
                            w1 = lds32(sc + (16 * mt + kr + 2) * 4);
                        } else {
                            w0 = lds32(sc + (16 * mt + (kr & ~1)) * 2) >> (16 * (kr & 1));
                            w1 = lds32(sc + (16 * mt + (kr & ~1) + 2) * 2) >> (16 * (kr & 1));
                        }
                        float acc[TILES][2];
#pragma unroll
                        for (int b = 0; b < BLOCKS; ++b) {
                            const uint32_t x0 = lds32(codes + 16 * mt * ROWB + k_at + (k_x0 ^ (b << 4)));
                            const uint32_t x1 = lds32(codes + (16 * mt + 2) * ROWB + k_at + (k_x1 ^ (b << 4)));
                            const uint32_t a[4] = {x0 & 0x0f0f0f0fu, x1 & 0x0f0f0f0fu, x0 >> 4 & 0x0f0f0f0fu, x1 >> 4 & 0x0f0f0f0fu};
                            const float s0 = __uint_as_float(__byte_perm(w0, 0, 0x4440 | b) * 0x100000u + 0x38000000u);
                            const float s1 = __uint_as_float(__byte_perm(w1, 0, 0x4440 | b) * 0x100000u + 0x38000000u);
#pragma unroll
                            for (int n = 0; n < TILES; ++n) {
                                float d[4];
                                mma_e4m3(d, a, q[n][b], init[n][b]);
                                // (rows g and g + 8; the low halves' columns join the high ones')
                                acc[n][0] = b ? fmaf(s0, d[0], acc[n][0]) : s0 * d[0];
                                acc[n][1] = b ? fmaf(s1, d[2], acc[n][1]) : s1 * d[2];
                                acc[n][0] = fmaf(s0, d[1], acc[n][0]);
                                acc[n][1] = fmaf(s1, d[3], acc[n][1]);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            s[n][2 * mt] = acc[n][0];
                            s[n][2 * mt + 1] = acc[n][1];
                        }
                    }
                    // ---- weights
                    const bool edge = (c + 1) * F4_KEYS > lowest;
                    uint32_t pk[QT][4];
                    float sum[TILES];
                    auto weights = [&]() {
                        float pr[TILES][4];
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            const float base = m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float y = fmaf(s[n][i], cq[n], -base);
                                if (edge && c * F4_KEYS + 16 * (i >> 1) + kr + 2 * (i & 1) >= limit[n]) y = -INFINITY;
                                pr[n][i] = ex2(y);
                            }
                            sum[n] = (pr[n][0] + pr[n][1]) + (pr[n][2] + pr[n][3]);
                        }
#pragma unroll
                        for (int j = 0; j < QT; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (TILES == 1) {   // p in two halves, in the two columns
                                    const float hi = bf16_lo(pack_bf16x2(pr[0][i], 0.f));
                                    pk[j][i] = pack_bf16x2(pr[0][i], pr[0][i] - hi);
                                } else {
                                    pk[j][i] = pack_bf16x2(pr[2 * j % TILES][i], pr[(2 * j + 1) % TILES][i]);
                                }
                            }
                    };
                    bool look = false;
#pragma unroll
                    for (int n = 0; n < TILES; ++n) look |= m[n] == -INFINITY;
                    look = __any_sync(0xffffffffu, look);
                    if (!look) {
                        weights();
#pragma unroll
                        for (int n = 0; n < TILES; ++n) look |= !(sum[n] <= F4_MOST);
                        look = __any_sync(0xffffffffu, look);
                    }
                    if (look) {
                        float f[TILES];
                        bool move = false;
#pragma unroll
                        for (int n = 0; n < TILES; ++n) {
                            float top = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float y = s[n][i] * cq[n];
                                if (!(edge && c * F4_KEYS + 16 * (i >> 1) + kr + 2 * (i & 1) >= limit[n])) top = fmaxf(top, y);
                            }
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                            f[n] = 1.f;
                            if (top > m[n] + 8.f) {
                                f[n] = ex2(m[n] - top);
                                m[n] = top;
                                l[n] *= f[n];
                                move = true;
                            }
                        }
                        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                            for (int j = 0; j < QT; ++j)
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const float fx = f[TILES == 1 ? 0 : (2 * j + (x & 1)) % TILES];
                                    z[j][x] *= fx;
#pragma unroll
                                    for (int i = 0; i < MT; ++i) o[i][j][x] *= fx;
                                }
                        }
                        weights();
                    }
#pragma unroll
                    for (int n = 0; n < TILES; ++n) l[n] += sum[n];
                    // ---- outputs: codes times scale in bf16 (exact), 8 times the scales' own sum taken off at the end
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t bq[QT][2];
#pragma unroll
                        for (int j = 0; j < QT; ++j) {
                            bq[j][0] = transpose_8x8(pk[j][2 * mt]);
                            bq[j][1] = transpose_8x8(pk[j][2 * mt + 1]);
                        }
                        uint32_t s2[2];
                        if (D == 128) {
                            const uint4 x = lds128(sc + L::SCALES + (16 * mt + 4 * t) * 4);
                            s2[0] = q4_scale2(__byte_perm(x.x, x.y, sel));
                            s2[1] = q4_scale2(__byte_perm(x.z, x.w, sel));
                        } else {
                            const uint2 x = lds64(sc + L::SCALES + (16 * mt + 4 * t) * 2);
                            s2[0] = q4_scale2(__byte_perm(x.x, 0, sel));
                            s2[1] = q4_scale2(__byte_perm(x.y, 0, sel));
                        }
                        const uint32_t off[2] = {s2[0] + 0x83808380u, s2[1] + 0x83808380u};   // -128 s
                        uint32_t v[4][D / 64];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (D == 128) {
                                const uint2 x = lds64(codes + 16 * mt * ROWB + v_at[i]);
                                v[i][0] = x.x;
                                v[i][D / 64 - 1] = x.y;
                            } else {
                                v[i][0] = lds32(codes + 16 * mt * ROWB + v_at[i]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < QT; ++j) mma_bf16(z[j], s2[0], s2[0], s2[1], s2[1], bq[j]);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            const uint32_t lo01 = __byte_perm(v[0][x], v[1][x], 0x5410), hi01 = __byte_perm(v[0][x], v[1][x], 0x7632);
                            const uint32_t lo23 = __byte_perm(v[2][x], v[3][x], 0x5410), hi23 = __byte_perm(v[2][x], v[3][x], 0x7632);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                auto value = [&](uint32_t word, int pair) {
                                    const uint32_t raw = (word >> (4 * j) & 0x000f000fu) | 0x43004300u;   // 128 + code
                                    return q4_value(raw, s2[pair], off[pair]);
                                };
                                const uint32_t a0 = value(lo01, 0), a1 = value(hi01, 0), a2 = value(lo23, 1), a3 = value(hi23, 1);
#pragma unroll
                                for (int y = 0; y < QT; ++y) mma_bf16(o[4 * x + j][y], a0, a1, a2, a3, bq[y]);
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + 8 * (L::EMPTY + slot));
                }
            }
            // ---- this warp's part of the piece, once the parts that were here have been read
            if (!__all_sync(0xffffffffu, ok) || (use > 0 && !__all_sync(0xffffffffu, wait(L::PE + buf, (use - 1) & 1)))) break;
            if (part) {
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], x);
                    const int row = 4 * n + t;
                    if (g == 0) sts_f2(sbase + L::ML + ((buf * W + warp) * ROWS + row) * 8, make_float2(m[n], l[n]));
                    const uint32_t at = sbase + L::PART + (buf * W + warp) * L::PART_WARP + row * L::PART_ROW;
                    const int j = n / 2, x = n & 1;
                    const float zz = 8.f * (TILES == 1 ? z[0][0] + z[0][1] : z[j][x]);
                    float y[D / 8];   // channels (D / 8) g ..
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        y[2 * i] = (TILES == 1 ? o[i][0][0] + o[i][0][1] : o[i][j][x]) - zz;
                        y[2 * i + 1] = (TILES == 1 ? o[i][0][2] + o[i][0][3] : o[i][j][2 + x]) - zz;
                    }
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        sts_f4(at + (((D / 32) * g + i) ^ t) * 16, make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8 * (L::PF + buf));
            // ---- one warp joins the parts
            if (pieces % W == (uint32_t)warp) {
                if (!__all_sync(0xffffffffu, wait(L::PF + buf, use & 1))) break;
                const bool closed = w.a == 0 && w.b == w.all;
                const int slot = 2 * blockIdx.x + (w.a > 0 ? 0 : 1);
                if (w.a == 0 && !closed && lane == 0) {
                    F4Join d;
                    d.n = w.n;
                    d.hk = w.hk;
                    d.row0 = w.first;
                    d.rows = w.rows;
                    d.pieces = 1 + (int)((w.rest + share - 1) / share);
                    p.join[blockIdx.x] = d;
                }
                constexpr int PIECES = D / 4, AT_ONCE = 32 / PIECES;
                const int piece = lane % PIECES;
                for (int r0 = 0; r0 < w.rows; r0 += AT_ONCE) {
                    const int row = r0 + lane / PIECES;
                    if (row >= w.rows) continue;
                    float top = -INFINITY, sum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    uint32_t who = run % W;
                    for (int i = 0; i < parts; ++i) {
                        top = fmaxf(top, lds_f2(sbase + L::ML + ((buf * W + who) * ROWS + row) * 8).x);
                        who = who + 1 == W ? 0 : who + 1;
                    }
                    const float ref = top == -INFINITY ? 0.f : top;
                    who = run % W;
                    for (int i = 0; i < parts; ++i) {
                        const float2 ml = lds_f2(sbase + L::ML + ((buf * W + who) * ROWS + row) * 8);
                        const float4 x = lds_f4(sbase + L::PART + (buf * W + who) * L::PART_WARP + row * L::PART_ROW + ((piece ^ (row & 3)) << 4));
                        const float f = ex2(ml.x - ref);
                        sum += f * ml.y;
                        acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
                        who = who + 1 == W ? 0 : who + 1;
                    }
                    if (closed) {
                        const int flat = w.first + row, tok = flat / p.G;
                        const size_t at = (size_t)(w.r.row0 + tok) * p.a.H_q + w.hk * p.G + (flat - tok * p.G);
                        if (w.r.keys - w.r.fresh + tok + 1 <= 0) sum = 0.f;   // no key, under a NaN scale too
                        const float inv = sum != 0.f ? 1.f / sum : 0.f;
                        const bool none = sum == 0.f;
                        *reinterpret_cast<uint2 *>(p.a.out + at * D + 4 * piece) =
                            none ? make_uint2(0, 0) : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                        if (piece == 0 && p.a.lse) p.a.lse[at] = none ? -INFINITY : (ref + lg2(sum)) * (1.f / LOG2E);
                    } else {
                        *reinterpret_cast<float4 *>(p.o + ((size_t)slot * F4_MAX_ROWS + row) * D + 4 * piece) = acc;
                        if (piece == 0) p.ml[slot * F4_MAX_ROWS + row] = make_float2(sum == 0.f ? -INFINITY : top, sum);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (L::PE + buf));
            }
            run += (uint32_t)n_chunks;
            ++pieces;
        }
    }
    if (!__all_sync(0xffffffffu, ok)) {
        set_status(KDA_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
        // let what is in flight land before the CTA leaves (bounded)
        for (int i = 0; i < W * S; ++i)
            for (uint32_t pp = 0; pp < 2; ++pp) mbar_wait(bar + 8 * (L::FULL + i), pp, 1u << 12);
    }
    __syncthreads();
}

// Joins the pieces of a unit that several CTAs worked on, in the order of the CTAs.
template <int D>
__global__ __launch_bounds__(128) void attn_q4_join_kernel(const F4Params p) {
    const int cta = blockIdx.x;
    grid_dep_wait();   // launched while the pieces are still being computed
    const F4Join d = p.join[cta];
    const int i = blockIdx.y * 128 + threadIdx.x, row = i / (D / 4), piece = i % (D / 4);
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

// ---------------------------------------------------------------- host side
int sm_count() {
    static int count[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!count[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        count[dev] = n < F4_MAX_CTAS ? n : F4_MAX_CTAS;
    }
    return count[dev];
}

// A cache's codes as (bytes of a row, row of a block, block and head), in boxes of at most 32 rows
template <int D>
cudaError_t codes_map(CUtensorMap *m, const uint8_t *base, const AttnQ4Args &a) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    const cudaError_t e = tma_encoder(&enc);
    if (e != cudaSuccess) return e;
    const cuuint64_t bs = 1ull << a.block_log2;
    const cuuint64_t dims[3] = {D / 2, bs, (cuuint64_t)a.num_blocks * a.H_kv};
    const cuuint64_t strides[2] = {D / 2, bs * q4_row_bytes(D)};
    const cuuint32_t box[3] = {D / 2, (cuuint32_t)(bs < F4_KEYS ? bs : F4_KEYS), 1}, one[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(base), dims, strides, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                           CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

size_t align256_f4(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, int ROWS>
cudaError_t run(const F4Params &p, int grid, cudaStream_t stream) {
    using L = F4Layout<D, ROWS>;
    CUtensorMap mk, mv;
    cudaError_t e = codes_map<D>(&mk, p.a.k, p.a);
    if (e == cudaSuccess) e = codes_map<D>(&mv, p.a.v, p.a);
    if (e != cudaSuccess) return e;
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    static bool ready[64] = {false};   // by device: the attribute is set once
    if (!ready[dev & 63]) {
        e = cudaFuncSetAttribute(attn_q4_few_kernel<D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::BYTES);
        if (e != cudaSuccess) return e;
        ready[dev & 63] = true;
    }
    attn_q4_few_kernel<D, ROWS><<<grid, L::THREADS, L::BYTES, stream>>>(mk, mv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, ROWS * (D / 4) / 128 > 0 ? ROWS * (D / 4) / 128 : 1);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_q4_join_kernel<D>, p);
}
}  // namespace

size_t attn_q4_few_workspace_bytes(int D) {
    return align256_f4(sizeof(F4Join) * F4_MAX_CTAS) + align256_f4(sizeof(float2) * 2 * F4_MAX_CTAS * F4_MAX_ROWS) +
           sizeof(float) * 2 * F4_MAX_CTAS * F4_MAX_ROWS * D;
}

cudaError_t launch_attn_q4_few(const AttnQ4Args &a, int most_rows, void *ws, cudaStream_t stream, int *launches) {
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    F4Params p;
    p.a = a;
    char *base = static_cast<char *>(ws);
    p.join = reinterpret_cast<F4Join *>(base);
    base += align256_f4(sizeof(F4Join) * F4_MAX_CTAS);
    p.ml = reinterpret_cast<float2 *>(base);
    base += align256_f4(sizeof(float2) * 2 * F4_MAX_CTAS * F4_MAX_ROWS);
    p.o = reinterpret_cast<float *>(base);
    p.c = a.scale * LOG2E;
    p.G = a.H_q / a.H_kv;
    p.most_rows = most_rows;
    p.unit_cost = 4;
    // rows a request has on average, or a single token's where the average is not this kernel's
    long long rows = ((long long)a.T + a.N - 1) / a.N * p.G;
    if (rows > most_rows) rows = p.G;
    *launches += 2;
    if (a.D == 64) return rows <= 4 ? run<64, 4>(p, sms, stream) : rows <= 8 ? run<64, 8>(p, sms, stream) : run<64, 16>(p, sms, stream);
    return rows <= 4 ? run<128, 4>(p, sms, stream) : rows <= 8 ? run<128, 8>(p, sms, stream) : run<128, 16>(p, sms, stream);
}

}  // namespace kda
