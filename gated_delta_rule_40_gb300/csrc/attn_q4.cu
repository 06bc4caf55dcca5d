// Causal softmax attention over a paged cache held in 4 bits (kda_attn_paged_q4).
//
// Requests with few query rows (new tokens x query heads of a group: decoded and drafted tokens) are bound by the
// cache's bytes, the others (prompts' chunks) by the products.  Two kernels, each of which finds its own requests
// among the lengths on the device: attn_q4_few.cu expands codes in registers, as operands of small products, and
// attn.cu's attn_kernel expands tiles of 128 keys into shared memory for tcgen05.  The second is launched while the
// first runs and takes over its SMs as they become free (in turn: 43.2 against 40.9 us for 100 decoded tokens with heads
// of 64, 165 against 162 us for a mixed call, but 197 against 201 us for chunks alone); where it finds nothing to do it costs 1
// to 4 us.  One more kernel joins what both have cut.
#include "attn.h"
#include "attn_q4_few.cuh"

namespace kda {
namespace {
// Rows of a request up to which it is one with few.  The kernel for few takes as long for each 16 rows more, the other
// one as long for any number up to 128.  128 requests over 4096 keys, 32 heads over 8, with 16 rows 174 against 327 us,
// with 32 324 against 328, with 64 623 against 335; over 1024 keys with 32 rows 101 against 142 us, with 64 176 against
// 146; a single request over 131072 keys with 32 rows 86 against 100 us, with 64 165 against 101.
constexpr int F4_MOST_ROWS = 32;
}  // namespace

size_t attn_q4_workspace_bytes(int D) { return attn_q4_few_workspace_bytes(D) + attn_workspace_bytes(D); }

cudaError_t launch_attn_q4(const AttnQ4Args &a, void *ws, cudaStream_t stream, int *launches) {
    const int G = a.H_q / a.H_kv;
    const bool few = G <= F4_MOST_ROWS, many = (long long)a.T * G > F4_MOST_ROWS;
    const F4Params p = attn_q4_few_params(a, F4_MOST_ROWS, ws);
    const int rows = attn_q4_few_rows(a, F4_MOST_ROWS);
    if (few) {
        const cudaError_t e = launch_attn_q4_few(p, rows, stream, launches);
        if (e != cudaSuccess) return e;
    }
    if (many) {
        AttnArgs b = {};
        b.q = a.q; b.k = reinterpret_cast<const uint16_t *>(a.k); b.v = reinterpret_cast<const uint16_t *>(a.v);
        b.out = a.out; b.lse = a.lse; b.cu = a.cu; b.table = a.table; b.lens = a.lens; b.scale = a.scale;
        b.N = a.N; b.B = 1; b.T = a.T; b.H_q = a.H_q; b.H_kv = a.H_kv; b.D = a.D;
        b.num_blocks = a.num_blocks; b.block_log2 = a.block_log2; b.max_blocks = a.max_blocks;
        return launch_attn_q4_many(b, F4_MOST_ROWS / G, few ? &p : nullptr, rows,
                                   static_cast<char *>(ws) + attn_q4_few_workspace_bytes(a.D), stream, launches);
    }
    return launch_attn_q4_few_join(p, rows, stream, launches);
}

}  // namespace kda
