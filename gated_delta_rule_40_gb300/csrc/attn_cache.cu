// The paged key/value cache of the softmax-attention layers: the layout of a serving step in it
// (block table, slot map, packed offsets) and the store of new keys and values.
#include "kda_common.cuh"

namespace kda {

// ---------------------------------------------------------------- page plan
// With c, a a request's cached and new tokens and bs the block size, it owns o = ceil(c / bs) table
// entries and takes w = ceil((c + a) / bs) - o from the free list, after those of the requests before
// it; a new token at position p has slot table[p / bs] bs + p % bs.  Both prefix sums (of a and of w)
// run over all requests, so every CTA computes them for itself, 1024 requests at a time, instead of
// waiting for another's: a few loads a thread.  Each CTA then writes its share of the tokens, whose
// new blocks it reads from the free list directly (an entry that another CTA writes is never read),
// and of the per-request outputs.  A new block begins with a new token, whose thread enters the block
// in the table; a block that cannot be had is entered as -1, so that no later step takes an old id that
// stood there for the request's own.  Latency is the bound: 3.6 us for 64 single tokens, 6.3 us for 2000
// requests with 66000.
constexpr int PP_THREADS = 1024;

struct PagePlanParams {
    const int32_t *cached, *fresh, *free_blocks, *free_start;
    int32_t *table, *cu, *lens, *slots, *positions, *free_next;
    int N, T, max_blocks, block_log2, num_free;
};

__global__ __launch_bounds__(PP_THREADS) void page_plan_kernel(const PagePlanParams p) {
    __shared__ long long s_cu[PP_THREADS + 1];   // first new token of each request of the group
    __shared__ int s_cached[PP_THREADS];
    __shared__ long long s_free[PP_THREADS];     // free-list index of each request's first new block
    __shared__ long long w_tok[32], w_blk[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bs = 1 << p.block_log2;
    // a negative place is one past the list's end too, where nothing is handed out
    const uint32_t start = (uint32_t)p.free_start[0];
    long long tok_base = 0, blk_base = start;
    int bad = 0;
    // this CTA's tokens
    const long long per = (p.T + (long long)gridDim.x - 1) / gridDim.x;
    const long long t0 = per * blockIdx.x, t1 = min(t0 + per, (long long)p.T);

    for (int n0 = 0; n0 < p.N; n0 += PP_THREADS) {
        const int n = n0 + tid;
        long long c = 0, a = 0;
        if (n < p.N) {
            c = p.cached[n];
            a = p.fresh[n];
            if (c < 0 || a < 0) bad = KDA_ERR_BAD_SEQLENS;
            c = max(c, 0ll);
            a = max(a, 0ll);
        }
        const long long owned = (c + bs - 1) >> p.block_log2, want = (c + a + bs - 1) >> p.block_log2;
        const long long take = max(min(want, (long long)p.max_blocks) - owned, 0ll);
        if (want > p.max_blocks) bad = KDA_ERR_BAD_SEQLENS;
        // inclusive prefix sums over the group
        long long st = a, sb = take;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, st, o), y = __shfl_up_sync(0xffffffffu, sb, o);
            if (lane >= o) {
                st += x;
                sb += y;
            }
        }
        __syncthreads();   // the previous group's tables have been read
        if (lane == 31) {
            w_tok[warp] = st;
            w_blk[warp] = sb;
        }
        __syncthreads();
        if (warp == 0) {
            long long x = w_tok[lane], y = w_blk[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) {
                    x += u;
                    y += v;
                }
            }
            w_tok[lane] = x;
            w_blk[lane] = y;
        }
        __syncthreads();
        const long long tok_end = tok_base + st + (warp ? w_tok[warp - 1] : 0);
        const long long first_blk = blk_base + sb - take + (warp ? w_blk[warp - 1] : 0);
        s_cu[tid + 1] = tok_end;
        if (tid == 0) s_cu[0] = tok_base;
        s_cached[tid] = (int)c;
        s_free[tid] = first_blk;
        if (n < p.N) {
            if (take > 0 && first_blk + take > p.num_free && !bad) bad = KDA_ERR_NO_BLOCKS;
            if (n % (int)gridDim.x == (int)blockIdx.x) {
                p.cu[n + 1] = (int)min(tok_end, 0x7fffffffll);
                p.lens[n] = (int)min(c + a, 0x7fffffffll);
            }
        }
        __syncthreads();
        tok_base += w_tok[31];
        blk_base += w_blk[31];
        // Enters a new block of the group's request r.  Without an id (-1) the entry names no block afterwards; one
        // that is negative does not anyway, and stays.
        auto enter = [&](int r, long long e, long long id) {
            int32_t *entry = p.table + (size_t)(n0 + r) * p.max_blocks + e;
            if (id >= 0 || *entry >= 0) *entry = (int)id;
        };
        // this CTA's tokens among the group's
        const long long lo = max(t0, s_cu[0]), hi = min(t1, s_cu[PP_THREADS]);
        for (long long t = lo + tid; t < hi; t += PP_THREADS) {
            int r = 0;   // last request of the group that starts at or before t
#pragma unroll
            for (int step = PP_THREADS / 2; step > 0; step >>= 1)
                if (s_cu[r + step] <= t) r += step;
            const long long cached = s_cached[r], pos = cached + (t - s_cu[r]);
            const long long e = pos >> p.block_log2, held = (cached + bs - 1) >> p.block_log2;
            long long id = -1;
            if (e < p.max_blocks) {
                const long long f = s_free[r] + (e - held);
                if (e < held) id = p.table[(size_t)(n0 + r) * p.max_blocks + e];
                else if (f < p.num_free) id = p.free_blocks[f];
                if (e >= held && (pos & (bs - 1)) == 0) enter(r, e, id);
                // an owned entry without a block (an earlier step could not have it), or such an id in the list
                if (id < 0 && (e < held || f < p.num_free)) bad = KDA_ERR_BAD_PAGES;
            }
            const long long slot = id < 0 ? -1 : (id << p.block_log2) + (pos & (bs - 1));
            if (slot > 0x7fffffffll) bad = KDA_ERR_BAD_PAGES;
            p.slots[t] = slot > 0x7fffffffll ? -1 : (int)slot;
            p.positions[t] = (int)min(pos, 0x7fffffffll);
        }
        // blocks whose first token is past T (reported below): entered all the same, a warp a request
        if (tok_base > p.T)
            for (int r = warp * gridDim.x + blockIdx.x; r < min(PP_THREADS, p.N - n0); r += 32 * gridDim.x) {
                const long long c = s_cached[r], held = (c + bs - 1) >> p.block_log2;
                const long long end = min((c + s_cu[r + 1] - s_cu[r] + bs - 1) >> p.block_log2, (long long)p.max_blocks);
                for (long long e = held + lane; e < end; e += 32) {
                    const long long f = s_free[r] + (e - held);
                    if (s_cu[r] + (e << p.block_log2) - c >= p.T) enter(r, e, f < p.num_free ? p.free_blocks[f] : -1);
                }
            }
    }
    // padding past the last token
    for (long long t = max(t0, tok_base) + tid; t < t1; t += PP_THREADS) p.slots[t] = p.positions[t] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        p.cu[0] = 0;
        p.free_next[0] = (int)(start <= (uint32_t)p.num_free ? min(blk_base, (long long)p.num_free) : start);
        if (start > (uint32_t)p.num_free) bad = KDA_ERR_NO_BLOCKS;
        if (tok_base > p.T) bad = KDA_ERR_BAD_SEQLENS;
    }
    if (bad) set_status(bad);
}

cudaError_t launch_page_plan(const int32_t *cached, const int32_t *fresh, const int32_t *free_blocks,
                             const int32_t *free_start, int32_t *table, int N, int T, int max_blocks, int block_log2,
                             int num_free, int32_t *cu, int32_t *lens, int32_t *slots, int32_t *positions,
                             int32_t *free_next, cudaStream_t stream) {
    PagePlanParams p;
    p.cached = cached; p.fresh = fresh; p.free_blocks = free_blocks; p.free_start = free_start;
    p.table = table; p.cu = cu; p.lens = lens; p.slots = slots; p.positions = positions; p.free_next = free_next;
    p.N = N; p.T = T; p.max_blocks = max_blocks; p.block_log2 = block_log2; p.num_free = num_free;
    const long long want = ((long long)T + PP_THREADS - 1) / PP_THREADS;
    const int grid = (int)(want < 1 ? 1 : want > 152 ? 152 : want);
    page_plan_kernel<<<grid, PP_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- cache write
// A row of one (token, head) is D bf16 = D / 8 units of 16 bytes; a thread moves one unit of k and the same
// one of v.  Neighbouring threads take neighbouring units, so loads are whole lines and stores whole rows of
// 128 or 256 bytes at the slot's place in each head.  DRAM is the bound: both loads go out before either
// store (32768 tokens x 8 heads of 128: 43.0 us on the GPU, 6.24 TB/s, a call 45 us; 45.6 us on the GPU with each
// store behind its own load; two or four units a thread 46.5 and 52.9 us, as a warp's accesses then skip lines).  The new
// keys and values are read once (streaming loads); the cache's lines stay, as attention reads them next.
__global__ __launch_bounds__(256) void kv_write_kernel(const uint4 *k, const uint4 *v, const int32_t *slots,
                                                       uint4 *k_cache, uint4 *v_cache, long long units, int per_token,
                                                       int per_row, int block_log2, int H_kv, long long num_slots) {
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= units) return;
    const long long t = u / per_token;
    const int in_token = (int)(u - t * per_token), h = in_token / per_row, x = in_token - h * per_row;
    const long long slot = slots[t];
    const uint4 a = __ldcs(k + u), b = __ldcs(v + u);
    if (slot < 0) return;
    if (slot >= num_slots) {
        set_status(KDA_ERR_BAD_PAGES);
        return;
    }
    const long long blk = slot >> block_log2, off = slot & ((1ll << block_log2) - 1);
    const long long dst = ((((blk * H_kv + h) << block_log2) + off) * per_row) + x;
    k_cache[dst] = a;
    v_cache[dst] = b;
}

cudaError_t launch_kv_write(const uint16_t *k, const uint16_t *v, const int32_t *slots, uint16_t *k_cache,
                            uint16_t *v_cache, int T, int H_kv, int D, int num_blocks, int block_log2,
                            cudaStream_t stream) {
    const int per_row = D / 8, per_token = H_kv * per_row;
    const long long units = (long long)T * per_token;
    kv_write_kernel<<<(unsigned)((units + 255) / 256), 256, 0, stream>>>(
        reinterpret_cast<const uint4 *>(k), reinterpret_cast<const uint4 *>(v), slots,
        reinterpret_cast<uint4 *>(k_cache), reinterpret_cast<uint4 *>(v_cache), units, per_token, per_row, block_log2,
        H_kv, (long long)num_blocks << block_log2);
    return cudaGetLastError();
}

}  // namespace kda
