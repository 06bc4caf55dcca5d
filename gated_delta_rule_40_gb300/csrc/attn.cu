// Causal softmax attention with grouped heads, over whole prompts (kda_attn_fwd) and over a paged
// cache (kda_attn_paged): s = scale q.k, o = sum exp(s - lse) v over the keys up to the query's own.
//
// Work.  A tile of queries is 128 rows: 128 / G tokens (rounded down) times the G query heads that
// share one key/value head, so that a key is read once for all of them and one decoded token with G
// heads needs one pass over its cache.  A unit is one or two such tiles of one (request, key/value
// head); it spans the tiles of 128 keys from the request's first to the last that its last token sees.
// The key tiles of all units, in order and with a constant for each unit's own cost (its queries' load, the
// start of its pipeline, its output), form one line that is cut into equal shares, one a CTA: a share may
// begin or end inside a unit, whose pieces attn_join_kernel then joins from (reference, sum, unnormalised
// output).  So a long cache with few rows, ragged lengths and the triangle of a causal prompt all divide
// evenly, without a schedule in memory: each CTA sums the requests' lengths itself.
//
// One CTA, 12 warps (an online softmax over steps of 64 keys, both products on the tensor cores):
//   loader    TMA: the query tiles (two slots) and key / value tiles of 128 keys (a ring) into
//             128-byte-swizzled shared memory; with pages, one box a page
//   cleaner   zeros in the value rows past a unit's last key, which may hold anything (another prompt, an
//             unused part of a block): p is 0 there, and 0 x NaN would be NaN
//   2 engines, each an issuing thread and four softmax warps on one query tile at a time (the two tiles of a
//             unit, or units of one tile in turn):
//     issuer  S = Q K^T (M = 128, N = 64) into one of two or three tensor-memory buffers, then O += P V
//             (P from tensor memory, V MN-major).  A step's scores are issued two or three steps ahead, so
//             that neither the tensor cores nor the softmax wait for the other's latency.  They overwrite the
//             weights that the output product BUFS steps before reads, and are issued behind it by the same thread
//             without waiting for it.  That rests on the tensor cores running one thread's products in the order
//             of their issue.  PTX promises that only for products with the same accumulator and shape, which
//             these are not, and no fence here adds to it; no run has shown another order.  Waiting for the
//             product takes 16384 tokens from 1.32 to 1.45 ms (spinning; 1.49 with try_wait), chunks among single
//             tokens from 127 to 142 us, decode from 347 to 350 us, and with heads of 64 a prompt of 2 x 4001
//             tokens from 98 to 100 us and decode (256 requests, 16 heads over 8) from 208 to 217 us.  (N = 128 would
//             need less of shared memory's bandwidth, which bounds a product of N = 64 to 48 cycles instead
//             of 32, but leaves room for one buffer only: 1.76 against 1.59 ms for a prompt of 16384 tokens.)
//     softmax a thread a row: s from tensor memory, p = 2^(s c - m c) with c = scale log2(e), the sum of p
//             in fp32, and p as bf16.  Tensor-core operands are bf16, so p is rounded to it: 2^-8 relative,
//             like the output's own rounding.  The reference m is the maximum of the row's first 64 keys
//             and moves only when a step's sum of p passes 2^16: a larger p costs no precision in floating
//             point, a common factor cancels in o, and neither the maximum nor a rescaling of O is needed
//             in most steps.
// Keys past a row's own position are masked in s.
//
// What bounds it, and what it measured (on the GPU, without a call's host side).  Prompts: the tensor cores, whose N = 64 products wait for shared
// memory (75 % of its wavefronts at 8192 tokens), and over long runs the power limit (1.7 GHz): 16384
// tokens x 32 heads over 8 in 1.31 to 1.34 ms, 1640 to 1680 TFLOP/s, where cuBLAS sustains 1705 on the same
// board; 20 packed prompts with 16384 tokens in 0.42 to 0.43 ms.  Heads of 64: the softmax's arithmetic, 2 x 4001
// tokens x 16 heads in 0.086 ms by itself, 0.093 to 0.10 ms behind hot calls.  Decode: DRAM, 256 requests with
// 2.2 GB of keys and values in 0.346 to 0.349 ms, 6.4 TB/s; one request over 131072 keys in 0.093 ms, 5.8 TB/s, of
// which the start and the joining take 10 us.  The ring's 160 KiB (heads of 128) cover DRAM's latency at the 45 GB/s
// that an SM gets of its bandwidth.  Decode with heads of 64 (a ring of 128 KiB): 256 requests, 16 heads over 8, with
// 1.1 GB in 0.208 ms, 5.3 TB/s.
//
// Every wait is bounded; a timeout records KDA_ERR_DEVICE_TIMEOUT and all roles stop.
#include "attn.h"
#include "kda_common.cuh"
#include "kda_tma.cuh"

namespace kda {

constexpr int AT_KEYS = 128;                 // keys a tile
constexpr int AT_ROWS = 128;                 // rows a query tile
constexpr long long AT_MAX_KEYS = 0x7fffff00;   // key positions, rounded up to a tile, stay below 2^31
constexpr int AT_THREADS = 384;              // 8 softmax warps, 2 issuers, loader, cleaner
constexpr int AT_ISSUER = 8, AT_LOADER = 10, AT_CLEANER = 11;   // warps
constexpr int AT_STEP = 64;                  // keys a softmax step
constexpr int AT_TILES = 2;                  // query tiles a unit: with one, every key tile is loaded twice as often
                                             // and one engine is idle (16384 tokens: 1.79 against 1.31 ms)
constexpr int AT_SHARE = 2;                  // key tiles a CTA has at least (4 decoded tokens over 1000 keys: 13 us
                                             // with 1 or 2, 16 with 3 or 4)
constexpr int AT_LEAST = 3;                  // tiles of a piece of a unit of two query tiles, at least
constexpr float AT_SLACK = 8.0f;             // log2 of how far a row's maximum may outgrow its reference in a step that
                                             // looks at it
constexpr float AT_MOST = 65536.0f;          // sum of a step's p that makes it look

template <int D, bool PAGED>
struct AttnLayout {
    static constexpr uint32_t TILE = AT_KEYS * D * 2;          // bytes of a query, key or value tile
    static constexpr int STAGES = D == 128 ? 5 : 8;            // key / value ring
    // A tile is made of 8-row x 64-channel swizzled blocks of 1 KiB.  A query tile, and a key or value tile of a
    // prompt, holds 64 channels of all rows, then the others; with pages, all channels of 8 rows, then the next
    // 8, so that a page, whatever its length, is one box.
    static constexpr uint32_t Q_HALF = AT_ROWS * 128;
    static constexpr uint32_t HALF = PAGED ? 1024 : AT_KEYS * 128;   // from a block to the other 64 channels'
    static constexpr uint32_t GROUP = PAGED ? 16 * D : 1024;         // from a block to the next 8 rows'
    static constexpr uint32_t Q = STAGES * TILE, BAR = Q + 2 * TILE;
    // Buffers of scores an engine has: what tensor memory holds beside two outputs of D columns
    static constexpr uint32_t BUFS = (512 - 2 * D) / (2 * AT_STEP) < 3 ? 2 : 3;
    // barriers: query tile loaded / free [slot]; scores ready, weights ready, output product done
    // [engine][buffer]; output read [engine]; key / value tile loaded / free, value tile to be cleaned loaded
    // [stage].  A step's scores are ready only after the output product BUFS steps before it, so that with one
    // barrier a buffer no wait can take an earlier phase for its own.
    enum { QF = 0, QE = 2, SF = 4, PF = SF + 2 * BUFS, PV = PF + 2 * BUFS, OE = PV + 2 * BUFS, KF = OE + 2,
           KE = KF + STAGES, VL = KF + 2 * STAGES, COUNT = KF + 3 * STAGES };
    static constexpr uint32_t SLOT = BAR + 8 * COUNT, FLAG = SLOT + 4, BYTES = BAR + 512 + 1024;
    static_assert(2 * D + 2 * AT_STEP * BUFS <= 512 && 8 * COUNT + 8 <= 512 && BYTES <= 232448, "attention shared memory");
};

// A unit cut by a share's end: its rows, and how many CTAs from this one on hold a piece of it.
struct JoinDesc {
    int row0, tokens[2], hk, pieces;
};

struct AttnParams {
    AttnArgs a;
    JoinDesc *join;   // NULL where no unit can be cut
    float2 *ml;       // [CTA][2][256] reference maximum (in log2 units) and sum of a piece's rows
    float *o;         // [CTA][2][D / 4][256][4] unnormalised outputs
    float c;          // scale log2(e), not negative
    int neg;          // the scale's sign
    bool whole;       // out is aligned to 32 bytes
    int G, tile_tokens;   // query heads a key/value head, tokens a tile
    int unit_cost;    // of a unit with two query tiles, in key tiles
};

// Sum of floor((a i + b) / m) over 0 <= i < n, a, m >= 1 (Euclid's descent on the lattice points under a
// line).  a n + b stays below 2^31 here: n <= 2^24 units, as a call has at most 2^31 rows, and after its
// reduction a < 128.
__host__ __device__ inline long long floor_sum(uint32_t n, uint32_t m, uint32_t a, long long b0) {
    long long sum = (long long)n * (b0 / m);
    uint32_t b = (uint32_t)(b0 % m);
    while (n > 0) {
        sum += (long long)n * (n - 1) / 2 * (a / m);
        a %= m;
        const uint32_t y = a * n + b;
        n = y / m;
        b = y % m;
        const uint32_t t = a;
        a = m;
        m = t;
        if (n > 0) {
            sum += (long long)n * (b / m);
            b %= m;
        }
    }
    return sum;
}

// One request: its rows, keys and units
struct Request {
    int row0, fresh, keys, units;
    int cost, least;   // of a unit: its cost beside its tiles, the fewest tiles of a piece
    __host__ __device__ void load(const AttnParams &p, int n) {
        if (p.a.cu) {
            row0 = p.a.cu[n];
            fresh = p.a.cu[n + 1] - row0;
            keys = p.a.lens ? p.a.lens[n] : fresh;
        } else {
            row0 = n * p.a.T;
            fresh = keys = p.a.T;
        }
        const int w = p.tile_tokens * AT_TILES;
        units = (fresh + w - 1) / w;
        cost = fresh > p.tile_tokens ? p.unit_cost : 0;
        least = fresh > p.tile_tokens ? AT_LEAST : 1;
    }
    // key tiles of the tokens up to (not including) token `end` of the request; at least one, for the
    // rows that see nothing
    __host__ __device__ int tiles_to(int end) const {
        const int seen = keys - fresh + min(end, fresh);
        return seen > AT_KEYS ? (seen + AT_KEYS - 1) / AT_KEYS : 1;
    }
    // A cut of a unit of n tiles at place x of its cost + n: there, or at its start or end where a piece would be
    // too short to be worth its joining
    __host__ __device__ int cut(int x, int n) const {
        return x - cost < least ? 0 : cost + n - x < least ? cost + n : x;
    }
    // length of the first u units (u <= units) of w tokens each: their key tiles and their costs
    // (not inlined: code that runs once is paid for by its fetching)
    __host__ __device__ __noinline__ long long prefix(int u, int w) const {
        long long sum = (long long)u * cost, first = keys - fresh;   // a unit has max(1, ceil((first + (j + 1) w) / 128)) tiles
        int full = u;
        if (u > 0 && u == units) {
            --full;
            sum += tiles_to(fresh);
        }
        int j0 = 0;   // units that see nothing at all or no more than one tile through a negative start
        if (first < 0) {
            j0 = (int)min((long long)full, (-first) / w);
            sum += j0;
            first += (long long)j0 * w;
            if (j0 < full && first < 0) {   // the unit that reaches the first key: it ends below w <= 256
                sum += max(1ll, (first + w + AT_KEYS - 1) / AT_KEYS);
                ++j0;
                first += w;
            }
        }
        return full > j0 ? sum + floor_sum(full - j0, AT_KEYS, w, first + w + AT_KEYS - 1) : sum;
    }
};

// The pieces of units in this CTA's share, in order
struct Walk {
    Request r;
    int n, hk, unit, at;
    long long left;
    // the current piece
    int a, b, all, token0, tokens[2];
    int end[2];      // steps of a query tile up to the piece's end
    int engine;      // of the first query tile
    long long line_end;   // place of the share's end in the unit's line
    __host__ __device__ void start(const Request &r_, int n_, int hk_, int unit_, int at_, long long left_) {
        engine = 1;
        tokens[1] = 0;
        n = n_; hk = hk_; unit = unit_; at = at_; left = left_;
        r = r_;
    }
    __host__ __device__ bool next(const AttnParams &p) {
        for (;;) {
            if (left <= 0) return false;
            if (unit >= r.units) {
                unit = 0;
                if (++hk == p.a.H_kv) {
                    hk = 0;
                    do r.load(p, ++n);
                    while (r.units == 0);
                }
            }
            token0 = unit * p.tile_tokens * AT_TILES;
            all = r.tiles_to(token0 + p.tile_tokens * AT_TILES);
            // from place `at` of the unit's cost + all
            const int whole = all + r.cost, from = r.cut(at, all), to = at + left >= whole ? whole : r.cut((int)(at + left), all);
            line_end = at + left;
            left = at + left >= whole ? at + left - whole : 0;
            a = max(from - r.cost, 0);
            b = max(to - r.cost, 0);
            at = 0;
            ++unit;
            if (b > a) break;   // nothing of this unit is left to the share
        }
        const int w = p.tile_tokens;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tokens[i] = max(0, min(w, r.fresh - token0 - i * w));
            const int seen = r.keys - r.fresh + token0 + i * w + tokens[i];
            end[i] = tokens[i] ? min(2 * b, seen > AT_STEP ? (seen + AT_STEP - 1) / AT_STEP : 1) : 0;
        }
        engine = tokens[1] ? 0 : engine ^ 1;
        return true;
    }
    __host__ __device__ bool active(int i) const { return end[i] > 2 * a; }
    // the query tile that engine e works on, or -1
    __host__ __device__ int tile_of(int e) const { return tokens[1] ? e : e == engine ? 0 : -1; }
    // whether the value rows of tile t do not end with it
    __host__ __device__ bool dirty(const AttnParams &p, int t) const { return keys(p) < (t + 1) * AT_KEYS; }
    // keys that the unit's last token sees
    __host__ __device__ int keys(const AttnParams &p) const {
        return max(0, r.keys - r.fresh + min(token0 + p.tile_tokens * AT_TILES, r.fresh));
    }
};

// One lane of a converged warp.  The tensor-core instructions take their operands from uniform registers:
// under this predicate, and with a warp index that is uniform to the compiler too, an issue costs about
// 65 cycles; under lane == 0 every operand is moved there first, about 100 cycles.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(mbar)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, int v,
                                            uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];\n" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(mbar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// One probe of a barrier's phase (the thread may sleep in it for a while)
__device__ __forceinline__ bool mbar_try(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
    return done != 0;
}

// 32 bytes to one place: a whole sector where the place is aligned to it
__device__ __forceinline__ void store_32_bytes(void *dst, const uint32_t *w, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <int D, bool PAGED>
__global__ __launch_bounds__(AT_THREADS, 1) void attn_kernel(const __grid_constant__ CUtensorMap tq,
                                                             const __grid_constant__ CUtensorMap tk,
                                                             const __grid_constant__ CUtensorMap tv,
                                                             const __grid_constant__ AttnParams p) {
    using L = AttnLayout<D, PAGED>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = aligned_smem<1024>(smem_raw);
    __shared__ long long s_warp[AT_THREADS / 32], s_x, s_head, s_at;
    __shared__ int s_n, s_unit;
    __shared__ Request s_req;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t sbase = smem_u32(sm), bar = sbase + L::BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::FLAG);
    const int nseq = p.a.cu ? p.a.N : p.a.B;
    grid_dep_launch();   // the joining kernel may come as soon as CTAs leave

    // barriers and tensor memory, under the latency of the lengths' loads
    bool bad = false;
    if (tid == 0) {
        if (p.join) p.join[blockIdx.x].pieces = 0;
        bad = p.a.cu && (p.a.cu[0] != 0 || (PAGED ? p.a.cu[p.a.N] > p.a.T : p.a.cu[p.a.N] != p.a.T));
    } else if (tid == 32) {
        for (int i = 0; i < L::COUNT; ++i)
            mbar_init(bar + 8 * i, i >= L::KE && i < L::VL ? 2 : (i >= L::PF && i < L::PV) || (i >= L::OE && i < L::KF) ? 4 : 1);
        mbar_fence_init();
        *abort_flag = 0;
        s_unit = 0;
    } else if (tid >= 64 && tid < 67) {
        prefetch_map(tid == 64 ? &tq : tid == 65 ? &tk : &tv);
    }
    if (warp == AT_LOADER) tmem_alloc(sbase + L::SLOT, 512);
    auto leave = [&]() {
        if (warp == AT_LOADER) tmem_dealloc(*reinterpret_cast<volatile uint32_t *>(sm + L::SLOT), 512);
    };

    // ---- this CTA's share: the length of all requests, then the request that holds the share's start
    long long total = 0, mine = 0, before = 0;
    Request mine_req;
    auto group = [&](int n0) {   // lengths of requests n0 + tid: this thread's, the ones before it, all
        const int n = n0 + tid;
        mine = 0;
        if (n < nseq) {
            mine_req.load(p, n);
            bool wrong = p.a.cu && p.a.cu[n + 1] < p.a.cu[n];
            if (PAGED)
                wrong |= mine_req.keys < 0 ||
                         mine_req.keys > min((long long)p.a.max_blocks << p.a.block_log2, AT_MAX_KEYS);
            bad |= wrong;
            if (!wrong) mine = mine_req.prefix(mine_req.units, p.tile_tokens * AT_TILES) * p.a.H_kv;
        }
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (nseq > AT_THREADS) __syncthreads();   // the last group's sums have been read
        if (lane == 31) s_warp[warp] = x;
        bad = __syncthreads_or(bad);
        long long sum = 0;
        before = x - mine;
#pragma unroll
        for (int w = 0; w < AT_THREADS / 32; ++w) {
            if (w < warp) before += s_warp[w];
            sum += s_warp[w];
        }
        return sum;
    };
    // 32-bit divisions wherever they do
    auto divide = [](long long a, long long b) {
        return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
    };
    tc_fence_before();
    // first pass: the sum of all; second pass, up to the group that holds the start (the first pass's only
    // group, mostly)
    long long share = 0, start = 0, left = 0, base = 0;
    bool found = false;
    for (int pass = 0; pass < 2 && !found; ++pass) {
        base = 0;
        for (int n0 = 0; !found && (n0 < nseq || n0 == 0); n0 += AT_THREADS) {
            const long long sum = group(n0);
            if (pass == 0) {
                total += sum;
                if (n0 + AT_THREADS < nseq) continue;
                if (bad) {
                    if (tid == 0) set_status(KDA_ERR_BAD_SEQLENS);
                    leave();
                    return;
                }
                share = max(divide(total + gridDim.x - 1, gridDim.x), (long long)AT_SHARE);
                start = share * blockIdx.x;
                left = min(share, total - start);
                if (left <= 0) {
                    leave();
                    return;
                }
                if (nseq > AT_THREADS) break;
            }
            if (start < base + sum) {
                found = true;
                if (start >= base + before && start < base + before + mine) {
                    s_n = n0 + tid;
                    s_x = start - (base + before);
                    s_head = divide(mine, p.a.H_kv);
                    s_req = mine_req;
                }
            }
            base += sum;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + L::SLOT);
    const uint32_t tS = tmem, tO = tmem + 2 * AT_STEP * L::BUFS;

    // the head and unit that hold place s_x of request s_n: every thread tries one unit, the last that starts at
    // or before it wins
    Walk w;
    {
        const Request r = s_req;
        const int wt = p.tile_tokens * AT_TILES;
        const int hk = (int)divide(s_x, s_head);
        long long x = s_x - hk * s_head;
        int unit = 0;
        if (r.units > 1) {
            const int step = (r.units + AT_THREADS - 1) / AT_THREADS, u = min(tid * step, r.units - 1);
            const long long at = r.prefix(u, wt);
            if (at <= x) atomicMax(&s_unit, u);
            __syncthreads();
            unit = s_unit;
            if (unit == u) s_at = at;
            __syncthreads();
            x -= s_at;
            for (int n; x >= (n = r.tiles_to((unit + 1) * wt) + r.cost); ++unit) x -= n;
        }
        w.start(r, s_n, hk, unit, (int)x, left);
    }

    // Bounded waits, of one thread or of a whole warp (whose lanes give up together).  The first probe is on its
    // own: for a phase that is complete already, which is the rule, it is all that runs.
    bool ok = true;
    constexpr uint32_t LIMIT = 1u << 22;
    auto wait_one = [&](int b, uint32_t parity) {
        if (mbar_try(bar + 8 * b, parity)) return true;
        for (uint32_t i = 0; i < LIMIT; ++i) {
            if (mbar_try(bar + 8 * b, parity)) return true;
            if ((i & 63) == 63 && *abort_flag) break;
        }
        return ok = false;
    };
    auto wait = [&](int b, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try(bar + 8 * b, parity))) return true;
        for (uint32_t i = 0; i < LIMIT; ++i) {
            if (__all_sync(0xffffffffu, mbar_try(bar + 8 * b, parity))) return true;
            if ((i & 63) == 63 && __any_sync(0xffffffffu, *abort_flag)) break;
        }
        return ok = false;
    };

    if (warp == AT_LOADER) {
        // ------------------------------------------------------------ loader
        uint32_t kv = 0, qu = 0;
        constexpr int HALVES = D / 64;
        // with pages: a tile is `boxes` boxes of `box` keys
        const int box = PAGED ? min(AT_KEYS, 1 << p.a.block_log2) : AT_KEYS, boxes = AT_KEYS / box;
        while (ok && w.next(p)) {
            const int keys = w.keys(p);
            // block id of this lane's box of tile t; looked at only when the tile is loaded, a tile later
            auto page = [&](int t) {
                if (!PAGED) return 0;
                const int key = t * AT_KEYS + lane * box;
                if (lane >= boxes || key >= keys || t >= w.b) return 0;
                return p.a.table[(size_t)w.n * p.a.max_blocks + (key >> p.a.block_log2)];
            };
            int id = page(w.a);
            auto queries = [&]() {
                for (int i = 0; i < 2; ++i) {
                    if (!w.active(i)) continue;
                    const uint32_t slot = qu & 1, u = qu >> 1;
                    ++qu;
                    if (u > 0 && !wait(L::QE + slot, (u - 1) & 1)) break;
                    if (lane == 0) {
                        const uint32_t qf = bar + 8 * (L::QF + slot);
                        mbar_expect_tx(qf, (uint32_t)(p.G * p.tile_tokens * 128 * HALVES));
                        for (int h = 0; h < HALVES; ++h)
                            tma_load_3d(sbase + L::Q + slot * L::TILE + h * L::Q_HALF, &tq, h * 64, w.hk * p.G,
                                        w.r.row0 + w.token0 + i * p.tile_tokens, qf);
                    }
                    __syncwarp();
                }
            };
            // the first queries go out at once; later ones follow the piece's first key tile, so that they wait
            // for their slot under its load
            const bool early = qu == 0;
            if (early) queries();
            for (int t = w.a; ok && t < w.b; ++t) {
                const int next_id = page(t + 1);
                if (PAGED && (id < 0 || id >= p.a.num_blocks)) {
                    set_status(KDA_ERR_BAD_PAGES);
                    id = p.a.num_blocks;   // past the tensor: zeros
                }
                const int n_box = PAGED ? max(0, min(boxes, (keys - t * AT_KEYS + box - 1) / box)) : 1;
                for (int part = 0; part < 2; ++part, ++kv) {
                    const uint32_t s = kv % L::STAGES, use = kv / L::STAGES;
                    if (use > 0 && !wait(L::KE + s, (use - 1) & 1)) break;
                    const uint32_t f = bar + 8 * ((part && w.dirty(p, t) ? L::VL : L::KF) + s);
                    if (lane == 0) mbar_expect_tx(f, (uint32_t)(n_box * box * 128 * HALVES));
                    __syncwarp();
                    const CUtensorMap *m = part ? &tv : &tk;
                    const uint32_t dst = sbase + s * L::TILE;
                    if (PAGED) {
                        const int off = (t * AT_KEYS + lane * box) & ((1 << p.a.block_log2) - 1);
                        if (lane < n_box)
                            tma_load_5d(dst + lane * (box / 8) * L::GROUP, m, 0, 0, 0, off / 8, id * p.a.H_kv + w.hk, f);
                    } else if (lane == 0) {
                        tma_load_4d(dst, m, 0, w.r.row0 + t * AT_KEYS, 0, w.hk, f);
                    }
                    if (t == w.a && part == 0 && !early) queries();
                }
                id = next_id;
            }
        }
    } else if (warp == AT_CLEANER) {
        // ------------------------------------------------------------ cleaner
        uint32_t kv = 0, uses = 0;   // ring entries so far; per stage, the parity of its value tiles cleaned
        while (ok && w.next(p)) {
            const int t = w.b - 1;
            kv += 2 * (uint32_t)(w.b - w.a);
            if (!w.dirty(p, t)) continue;
            const uint32_t stage = (kv - 1) % L::STAGES;
            if (!wait(L::VL + stage, (uses >> stage) & 1)) break;
            uses ^= 1u << stage;
            unsigned char *v = sm + stage * L::TILE;
            for (int u = max(w.keys(p) - t * AT_KEYS, 0) * 8 + lane; u < AT_KEYS * 8; u += 32)
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    *reinterpret_cast<uint4 *>(v + (u >> 6) * L::GROUP + h * L::HALF + (u & 63) * 16) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8 * (L::KF + stage));
        }
    } else if (warp >= AT_ISSUER) {
        // ------------------------------------------------------------ issuing thread of engine e
        const int e = warp - AT_ISSUER;
        if (elect_lane()) {
            constexpr uint32_t id_s = idesc_bf16(128, AT_STEP), id_o = idesc_bf16(128, D) | (1u << 16);
            constexpr uint32_t HALF_STEP = AT_STEP / 8 * L::GROUP;   // bytes between a tile's two steps
            const uint32_t s_at = tS + AT_STEP * L::BUFS * e, o_at = tO + D * e;
            // ring positions of the next key and value tile
            uint32_t ks = 0, kp = 0, vs = 1, vp = 0;
            auto advance = [](uint32_t &stage, uint32_t &phase) {
                stage += 2;
                if (stage >= L::STAGES) {
                    stage -= L::STAGES;
                    phase ^= 1;
                }
            };
            uint32_t qu = 0, steps = 0, jobs = 0;   // query tiles of both engines, this engine's steps and jobs so far
            while (ok && w.next(p)) {
                const int i = w.tile_of(e);
                const bool mine = i >= 0 && w.active(i);
                uint32_t slot = 0;
                for (int k = 0; k < 2; ++k)
                    if (w.active(k)) {
                        if (mine && k == i) {
                            slot = qu & 1;
                            wait_one(L::QF + slot, (qu >> 1) & 1);
                        }
                        ++qu;
                    }
                const int s0 = 2 * w.a, s1 = mine ? w.end[i] : s0;
                const uint64_t dq = umma_desc(sbase + L::Q + slot * L::TILE, 16, 1024);
                // scores of step s
                auto scores = [&](int s) {
                    const uint32_t buf = (steps + (s - s0)) % L::BUFS;
                    if ((s & 1) == 0 && !wait_one(L::KF + ks, kp)) return;
                    tc_fence_after();
                    const uint64_t dk = umma_desc(sbase + ks * L::TILE + (s & 1) * HALF_STEP, 16, L::GROUP);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t to_q = (uint64_t)(((k >> 2) * L::Q_HALF + (k & 3) * 32) >> 4);
                        const uint64_t to_k = (uint64_t)(((k >> 2) * L::HALF + (k & 3) * 32) >> 4);
                        umma_bf16(s_at + AT_STEP * buf, dq + to_q, dk + to_k, id_s, k > 0 ? 1u : 0u);
                    }
                    umma_commit(bar + 8 * (L::SF + L::BUFS * e + buf));
                    if (s + 1 == s1) umma_commit(bar + 8 * (L::QE + slot));
                    if ((s & 1) || s + 1 == s1) {
                        umma_commit(bar + 8 * (L::KE + ks));
                        advance(ks, kp);
                    }
                };
                for (int s = s0; ok && s < s1 && s < s0 + (int)L::BUFS; ++s) scores(s);
                for (int s = s0; ok && s < s1; ++s) {
                    const uint32_t n = steps + (s - s0), buf = n % L::BUFS;
                    if ((s & 1) == 0 && !wait_one(L::KF + vs, vp)) break;
                    if (s == s0 && jobs > 0 && !wait_one(L::OE + e, (jobs - 1) & 1)) break;
                    if (!wait_one(L::PF + L::BUFS * e + buf, (n / L::BUFS) & 1)) break;
                    tc_fence_after();
                    const uint64_t dv = umma_desc(sbase + vs * L::TILE + (s & 1) * HALF_STEP, L::HALF, L::GROUP);
#pragma unroll
                    for (int k = 0; k < AT_STEP / 16; ++k)
                        umma_bf16_ta(o_at, s_at + AT_STEP * buf + 8 * k, dv + (uint64_t)(k * (2 * L::GROUP >> 4)), id_o,
                                     s > s0 || k > 0 ? 1u : 0u);
                    umma_commit(bar + 8 * (L::PV + L::BUFS * e + buf));
                    if ((s & 1) || s + 1 == s1) {
                        umma_commit(bar + 8 * (L::KE + vs));
                        advance(vs, vp);
                    }
                    // the next scores take this step's buffer behind its product (see "issuer" at the top)
                    tc_fence_before();
                    if (s + (int)L::BUFS < s1) scores(s + L::BUFS);
                }
                // tiles of the piece that this engine has no part in
                for (int t = (s1 + 1) >> 1; ok && t < w.b; ++t) {
                    if (!wait_one(L::KF + ks, kp)) break;
                    mbar_arrive(bar + 8 * (L::KE + ks));
                    advance(ks, kp);
                    if (!wait_one(L::KF + vs, vp)) break;
                    mbar_arrive(bar + 8 * (L::KE + vs));
                    advance(vs, vp);
                }
                steps += (uint32_t)(s1 - s0);
                jobs += mine ? 1 : 0;
            }
            if (!ok || *abort_flag) {
                *abort_flag = 1;
                // let what is in flight land before the CTA releases tensor memory (bounded)
                for (int i = 0; i < L::COUNT; ++i)
                    for (uint32_t pp = 0; pp < 2; ++pp) mbar_wait(bar + 8 * i, pp, 1u << 12);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax of engine e
        const int e = warp >> 2, row = (warp & 3) * 32 + lane, tok = row / p.G, g = row - tok * p.G;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tS + AT_STEP * L::BUFS * e + lane_off, o_at = tO + D * e + lane_off;
        uint32_t ns = 0;   // steps so far: phases of S, P and PV
        // A negative scale: the sign goes into the factor of p with heads of 64, and into the scores, as they are read,
        // with heads of 128.  (2 x 4001 tokens x 16 heads of 64: 98 against 103 us; with heads of 128 the factor costs
        // prompts 0 to 2 % and pages 4 %.)
        constexpr bool FOLD = D == 64;
        const float c = p.c, factor = FOLD && p.neg ? -c : c;
        const uint32_t sign = FOLD && p.neg ? 0x80000000u : 0u, nothing = 0xff800000u ^ sign;   // -infinity
        while (ok && w.next(p)) {
            const bool closed = w.a == 0 && w.b == w.all;
            if (tid == 0 && w.a == 0 && !closed) {
                JoinDesc d;
                d.row0 = w.r.row0 + w.token0;
                d.tokens[0] = w.tokens[0];
                d.tokens[1] = w.tokens[1];
                d.hk = w.hk;
                // the shares' ends in the rest of the unit, the first of them this one's, that cut it
                d.pieces = 2 + (int)((w.all + w.r.cost - w.r.least - w.line_end) / share);
                p.join[blockIdx.x] = d;
            }
            const int i = w.tile_of(e);
            if (i < 0) continue;
            const bool real = tok < w.tokens[i];
            const bool warp_real = __any_sync(0xffffffffu, real);
            // keys this row sees; rows that stand for nothing see all, so that they need no mask
            const int limit = real ? w.r.keys - w.r.fresh + w.token0 + i * p.tile_tokens + tok + 1 : 0x7fffffff;
            float m = -INFINITY, l = 0.f;   // reference maximum of s, sum of p
            for (int s = 2 * w.a; ok && s < w.end[i]; ++s, ++ns) {
                const uint32_t buf = ns % L::BUFS;
                if (!wait(L::SF + L::BUFS * e + buf, (ns / L::BUFS) & 1)) break;
                if (warp_real) {
                    tc_fence_after();
                    uint32_t x[2][32], pk[2][16];
                    float2 sum;
#pragma unroll
                    for (int b = 0; b < 2; ++b) tmem_ld32_nowait(s_at + AT_STEP * buf + 32 * b, x[b]);
                    tmem_wait_ld();
                    if (!FOLD && p.neg) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[b][j] ^= 0x80000000u;
                    }
                    const int seen = limit - s * AT_STEP;   // columns of this step that the row sees
                    if (__any_sync(0xffffffffu, seen < AT_STEP)) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (32 * b + j >= seen) x[b][j] = nothing;
                    }
                    auto weights = [&]() {
                        const float base = m == -INFINITY ? 0.f : m * c;
                        const float2 c2 = make_float2(factor, factor), b2 = make_float2(-base, -base);
                        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                float2 y = __ffma2_rn(make_float2(__uint_as_float(x[b][j]), __uint_as_float(x[b][j + 1])), c2, b2);
                                y.x = ex2(y.x);
                                y.y = ex2(y.y);
                                part[(j >> 1) & 1] = __fadd2_rn(part[(j >> 1) & 1], y);
                                pk[b][j >> 1] = pack_bf16x2(y.x, y.y);
                            }
                        sum = __fadd2_rn(part[0], part[1]);
                    };
                    // (rows that stand for nothing hold what was in shared memory, and have no say)
                    bool look = __any_sync(0xffffffffu, real && m == -INFINITY);
                    if (!look) {
                        weights();
                        // written on trust: the check's latency runs under the store's
#pragma unroll
                        for (int b = 0; b < 2; ++b) tmem_st16(s_at + AT_STEP * buf + 16 * b, pk[b]);
                        look = __any_sync(0xffffffffu, real && !(sum.x + sum.y <= AT_MOST));
                    }
                    if (look) {
                        float mx[4];
                        auto score = [&](int j) { return __uint_as_float(x[j >> 5][j & 31] ^ sign); };
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            mx[b] = fmaxf(score(16 * b), score(16 * b + 1));
#pragma unroll
                            for (int j = 2; j < 16; j += 2) mx[b] = fmaxf(fmaxf(mx[b], score(16 * b + j)), score(16 * b + j + 1));
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        const bool grow = real && (top - m) * c > AT_SLACK;   // the first step's m is -infinity
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((m - top) * c) : 1.f;
                            if (grow) m = top;
                            l *= f;
                            if (s > 2 * w.a) {
                                if (!wait(L::PV + L::BUFS * e + (ns - 1) % L::BUFS, ((ns - 1) / L::BUFS) & 1)) break;
                                tc_fence_after();
#pragma unroll 1
                                for (int b = 0; b < D / 16; ++b) {
                                    uint32_t y[16];
                                    tmem_ld16_nowait(o_at + 16 * b, y);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                                    tmem_st16(o_at + 16 * b, y);
                                }
                            }
                        }
                        weights();
                        tmem_wait_st();
#pragma unroll
                        for (int b = 0; b < 2; ++b) tmem_st16(s_at + AT_STEP * buf + 16 * b, pk[b]);
                    }
                    l += sum.x + sum.y;
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (L::PF + L::BUFS * e + buf));
            }
            if (!ok) break;
            // ---- the piece's rows: final ones go out, others to the workspace
            if (w.active(i)) {
                if (!wait(L::PV + L::BUFS * e + (ns - 1) % L::BUFS, ((ns - 1) / L::BUFS) & 1)) break;
                tc_fence_after();
            }
            if (w.tokens[i] && warp_real) {
                const long long out_row = ((long long)w.r.row0 + w.token0 + i * p.tile_tokens + tok) * p.a.H_q + w.hk * p.G + g;
                const int piece = 2 * blockIdx.x + (w.a > 0 ? 0 : 1), prow = i * AT_ROWS + row;
                const bool any = w.active(i);
                if (limit <= 0) l = 0.f;   // no key: 0 and -infinity, under a NaN scale too
                const float inv = l != 0.f ? 1.f / l : 0.f;
                const float base = m == -INFINITY ? 0.f : m * c;
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    uint32_t y[2][32];
                    if (any) {
                        tmem_ld32_nowait(o_at + 64 * b, y[0]);
                        tmem_ld32_nowait(o_at + 64 * b + 32, y[1]);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; ++j) y[j >> 5][j & 31] = 0;
                    }
                    if (real && closed) {
                        uint32_t o[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = l != 0.f ? pack_bf16x2(__uint_as_float(y[j >> 4][(2 * j) & 31]) * inv,
                                                          __uint_as_float(y[j >> 4][(2 * j + 1) & 31]) * inv) : 0u;
#pragma unroll
                        for (int j = 0; j < 4; ++j) store_32_bytes(p.a.out + out_row * D + 64 * b + 16 * j, o + 8 * j, p.whole);
                    } else if (real) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            *reinterpret_cast<uint4 *>(p.o + (((size_t)piece * (D / 4) + 16 * b + j) * 256 + prow) * 4) =
                                make_uint4(y[j >> 3][(4 * j) & 31], y[j >> 3][(4 * j + 1) & 31], y[j >> 3][(4 * j + 2) & 31],
                                           y[j >> 3][(4 * j + 3) & 31]);
                    }
                }
                if (real) {
                    if (!closed) p.ml[(size_t)piece * 256 + prow] = make_float2(l != 0.f ? base : -INFINITY, l);
                    else if (p.a.lse) p.a.lse[out_row] = l != 0.f ? (base + lg2(l)) * (1.f / LOG2E) : -INFINITY;
                }
            }
            if (w.active(i)) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (L::OE + e));
            }
        }
    }
    if (!ok) {
        set_status(KDA_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == AT_LOADER) tmem_dealloc(tmem, 512);
}

// Joins the pieces of a unit that several CTAs worked on: with M the largest reference maximum,
// o = sum 2^(m - M) O / sum 2^(m - M) l.  Piece 0 is the opening CTA's second slot, the following ones the
// first slots of the CTAs after it, always in that order, so that a call gives the same bits again.  A thread takes 8
// channels of one row; the pieces are laid out with rows innermost, so a warp's loads are whole lines.  Bound by
// latency, and by L2 where every share cuts a unit of 256 rows (39 MB, 8 us); 2 us for a few decoded tokens.
template <int D>
__global__ __launch_bounds__(256, 4) void attn_join_kernel(const AttnParams p) {
    const int cta = blockIdx.x;
    grid_dep_wait();   // launched while the pieces are still being computed
    const JoinDesc d = p.join[cta];
    if (d.pieces == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int prow = blockIdx.y * 32 + lane, i = prow / AT_ROWS, row = prow % AT_ROWS;
    const int tok = row / p.G, g = row - tok * p.G;
    if (tok >= d.tokens[i]) return;
    auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * cta + 1 : 2 * (cta + k)); };
    const long long out_row = ((long long)d.row0 + i * p.tile_tokens + tok) * p.a.H_q + d.hk * p.G + g;
    const int c8 = blockIdx.z * 8 + warp;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f, M = -INFINITY;
    // four pieces at a time, so that their loads are in flight together
    for (int k0 = 0; k0 < d.pieces; k0 += 4) {
        float2 ml[4];
        float4 u[4], v[4];
        float top = M;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            u[k] = v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + k < d.pieces) {
                ml[k] = p.ml[slot(k0 + k) * 256 + prow];
                const float4 *src = reinterpret_cast<const float4 *>(p.o) + (slot(k0 + k) * (D / 4) + 2 * c8) * 256 + prow;
                u[k] = src[0];
                v[k] = src[256];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
        const float ref = top == -INFINITY ? 0.f : top, f0 = ex2(M - ref);
        l *= f0;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= f0;
        M = top;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = ex2(ml[k].x - ref);
            l += f * ml[k].y;
            o[0] += f * u[k].x; o[1] += f * u[k].y; o[2] += f * u[k].z; o[3] += f * u[k].w;
            o[4] += f * v[k].x; o[5] += f * v[k].y; o[6] += f * v[k].z; o[7] += f * v[k].w;
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<uint4 *>(p.a.out + out_row * D + 8 * c8) =
        make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                   pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    if (c8 == 0 && p.a.lse) p.a.lse[out_row] = l != 0.f ? (M + lg2(l)) * (1.f / LOG2E) : -INFINITY;
}

// ---------------------------------------------------------------- host side
namespace {
constexpr int AT_MAX_CTAS = 160;

int sm_count() {
    static int count[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!count[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        count[dev] = n < AT_MAX_CTAS ? n : AT_MAX_CTAS;
    }
    return count[dev];
}

// A bf16 tensor of n dimensions, the first of channels, with the others' strides in elements, in 128-byte
// swizzled boxes
cudaError_t tensor_map(CUtensorMap *m, const void *base, int n, const long long *sizes, const long long *strides,
                       const int *boxes) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    const cudaError_t e = tma_encoder(&enc);
    if (e != cudaSuccess) return e;
    cuuint64_t dims[5], bytes[4];
    cuuint32_t box[5], one[5];
    for (int i = 0; i < n; ++i) {
        dims[i] = (cuuint64_t)sizes[i];
        box[i] = (cuuint32_t)boxes[i];
        one[i] = 1;
        if (i > 0) bytes[i - 1] = (cuuint64_t)strides[i - 1] * 2;
    }
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)n, const_cast<void *>(base), dims, bytes, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

size_t align256_at(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, bool PAGED>
cudaError_t run(const AttnParams &p, int grid, cudaStream_t stream) {
    using L = AttnLayout<D, PAGED>;
    const AttnArgs &a = p.a;
    const long long rows = (long long)a.B * a.T;
    CUtensorMap mq, mk, mv;
    cudaError_t e;
    {   // (channel, head, row)
        const long long size[3] = {D, a.H_q, rows}, stride[2] = {D, (long long)a.H_q * D};
        const int box[3] = {64, p.G, p.tile_tokens};
        if ((e = tensor_map(&mq, a.q, 3, size, stride, box)) != cudaSuccess) return e;
    }
    for (int i = 0; i < 2; ++i) {
        const void *base = i ? a.v : a.k;
        CUtensorMap *m = i ? &mv : &mk;
        if (PAGED) {   // (64 channels, 8 rows, channel halves, groups of 8 rows in a block, block and head)
            const int bs = 1 << a.block_log2;
            const long long size[5] = {64, 8, D / 64, bs / 8, (long long)a.num_blocks * a.H_kv};
            const long long stride[4] = {D, 64, 8 * D, (long long)bs * D};
            const int box[5] = {64, 8, D / 64, (bs < AT_KEYS ? bs : AT_KEYS) / 8, 1};
            e = tensor_map(m, base, 5, size, stride, box);
        } else {   // (64 channels, row, channel halves, head)
            const long long size[4] = {64, rows, D / 64, a.H_kv}, stride[3] = {(long long)a.H_kv * D, 64, D};
            const int box[4] = {64, AT_KEYS, D / 64, 1};
            e = tensor_map(m, base, 4, size, stride, box);
        }
        if (e != cudaSuccess) return e;
    }
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    static bool ready[64] = {false};   // by device: the attributes are set once
    if (!ready[dev & 63]) {
        e = cudaFuncSetAttribute(attn_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::BYTES);
        if (e != cudaSuccess) return e;
        // the same split of an SM's memory for both kernels, so that it is not rearranged between them
        e = cudaFuncSetAttribute(attn_join_kernel<D>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        ready[dev & 63] = true;
    }
    attn_kernel<D, PAGED><<<grid, AT_THREADS, L::BYTES, stream>>>(mq, mk, mv, p);
    if ((e = cudaGetLastError()) != cudaSuccess || !p.join) return e;
    cudaLaunchConfig_t cfg = {};
    // rows that a unit can have: a tile's, and those of the next one behind it
    const int tokens = a.T < p.tile_tokens * AT_TILES ? a.T : p.tile_tokens * AT_TILES;
    const int unit_rows = tokens <= p.tile_tokens ? tokens * p.G : AT_ROWS + (tokens - p.tile_tokens) * p.G;
    cfg.gridDim = dim3(grid, (unit_rows + 31) / 32, D / 64);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, p);
}
}  // namespace

// A unit of two query tiles is cut into pieces of AT_LEAST key tiles or more, one of a single query tile anywhere;
// a prompt of up to 128 / G tokens has one key tile.  So prompts below 2 AT_LEAST key tiles are never cut, and
// need neither workspace nor the second kernel: 3 us on the GPU and 2 us of the host's.
bool attn_may_cut(const AttnArgs &a) { return a.lens || a.T > (2 * AT_LEAST - 1) * AT_KEYS; }

size_t attn_workspace_bytes(int D) {
    return align256_at(sizeof(JoinDesc) * AT_MAX_CTAS) + align256_at(sizeof(float2) * 256 * 2 * AT_MAX_CTAS) +
           sizeof(float) * 256 * D * 2 * AT_MAX_CTAS;
}

cudaError_t launch_attn(const AttnArgs &a, void *ws, cudaStream_t stream, int *launches) {
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    AttnParams p;
    p.a = a;
    const bool cut = attn_may_cut(a);
    char *base = static_cast<char *>(ws);
    p.join = cut ? reinterpret_cast<JoinDesc *>(base) : nullptr;
    base += align256_at(sizeof(JoinDesc) * AT_MAX_CTAS);
    p.ml = reinterpret_cast<float2 *>(base);
    base += align256_at(sizeof(float2) * 256 * 2 * AT_MAX_CTAS);
    p.o = reinterpret_cast<float *>(base);
    p.neg = a.scale < 0.f;
    p.whole = ((uintptr_t)a.out & 31u) == 0;
    // a scale of 0 keeps a vanishing factor instead: the masked scores' -infinity x 0 would be NaN.  A NaN stays one.
    p.c = fabsf(a.scale) * LOG2E;
    if (p.c < 1e-36f) p.c = 1e-36f;
    p.G = a.H_q / a.H_kv;
    p.tile_tokens = AT_ROWS / p.G;
    p.unit_cost = a.D == 128 ? 3 : 2;   // about 4 us, measured on packed prompts (a tile 1.3 us)
    *launches = cut ? 2 : 1;
    if (a.lens) return a.D == 64 ? run<64, true>(p, sms, stream) : run<128, true>(p, sms, stream);
    return a.D == 64 ? run<64, false>(p, sms, stream) : run<128, false>(p, sms, stream);
}

}  // namespace kda
