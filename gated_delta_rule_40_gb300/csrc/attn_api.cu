// C-ABI entry points of the softmax-attention serving operators: argument validation and launches.
// See include/kda.h for the contract.
#include "attn.h"
#include "kda_common.cuh"

namespace kda {
cudaError_t launch_page_plan(const int32_t *cached, const int32_t *fresh, const int32_t *free_blocks,
                             const int32_t *free_start, int32_t *table, int N, int T, int max_blocks, int block_log2,
                             int num_free, int32_t *cu, int32_t *lens, int32_t *slots, int32_t *positions,
                             int32_t *free_next, cudaStream_t stream);
cudaError_t launch_kv_write(const uint16_t *k, const uint16_t *v, const int32_t *slots, uint16_t *k_cache,
                            uint16_t *v_cache, int T, int H_kv, int D, int num_blocks, int block_log2,
                            cudaStream_t stream);
void set_last_launches(int n);
cudaError_t ws_alloc(void **p, size_t bytes, cudaStream_t stream);
cudaError_t ws_free(void *p, cudaStream_t stream);
void timing_begin(cudaStream_t s);
void timing_mark(const char *name, cudaStream_t s);
}  // namespace kda

namespace {
bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Every int32 array (or NULL) starts on 4 bytes
template <typename... P>
bool ints_aligned(const P *...p) {
    return (... && aligned(p, 4));
}

// log2 of a supported block size, or -1
int block_log2(int size) {
    for (int s = 4; s <= 10; ++s)
        if (size == 1 << s) return s;
    return -1;
}

bool heads_ok(int H_q, int H_kv) { return H_q > 0 && H_kv > 0 && H_q % H_kv == 0 && H_q / H_kv <= 128; }
bool cache_ok(int num_blocks, int log2) { return num_blocks >= 0 && ((long long)num_blocks << log2) <= 0x7fffffffLL; }

int finish(cudaError_t e, const char *name, cudaStream_t stream) {
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    kda::timing_mark(name, stream);
    kda::set_last_launches(1);
    return KDA_OK;
}
int nothing_to_do() {
    kda::set_last_launches(0);
    return KDA_OK;
}

// Tensors shared by the two attention calls; work items carry 32-bit indices
int validate_attn(const kda::AttnArgs &a) {
    if (a.D != 64 && a.D != 128) return KDA_ERR_UNSUPPORTED;
    if (a.B < 0 || a.T < 0 || a.N < 0 || !heads_ok(a.H_q, a.H_kv)) return KDA_ERR_INVALID_ARG;
    const long long tokens = (long long)a.B * a.T;
    if (tokens * a.H_q > 0x7fffffffLL || (long long)(a.cu ? a.N : a.B) * a.H_q > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
    if (tokens == 0) return KDA_OK;
    if (!a.q || !a.k || !a.v || !a.out) return KDA_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4) ||
        !ints_aligned(a.cu, a.table, a.lens))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Runs the kernels in the given workspace, or in one from the library's pool
int attend(const kda::AttnArgs &a, bool own_ws, void *ws, size_t ws_bytes, cudaStream_t stream) {
    const size_t need = kda::attn_workspace_bytes(a.D);
    const bool given = !own_ws;
    own_ws = own_ws && kda::attn_may_cut(a);
    if (own_ws) {
        if (kda::ws_alloc(&ws, need, stream) != cudaSuccess) return KDA_ERR_CUDA;
    } else if (given && (!ws || !aligned(ws, 256) || ws_bytes < need)) {
        return KDA_ERR_WORKSPACE;
    }
    int launches = 0;
    kda::timing_begin(stream);
    const cudaError_t e = kda::launch_attn(a, ws, stream, &launches);
    int rc = finish(e, "attn_kernel", stream);
    if (rc == KDA_OK) kda::set_last_launches(launches);
    if (own_ws && kda::ws_free(ws, stream) != cudaSuccess && rc == KDA_OK) rc = KDA_ERR_CUDA;
    return rc;
}

int prompt(const kda_bf16_t *q, const kda_bf16_t *k, const kda_bf16_t *v, float scale, const int32_t *cu_seqlens, int N,
           int B, int T, int H_q, int H_kv, int D, kda_bf16_t *out, float *lse, bool own_ws, void *ws, size_t ws_bytes,
           cudaStream_t stream) {
    kda::AttnArgs a = {};
    a.q = q; a.k = k; a.v = v; a.out = out; a.lse = lse; a.cu = cu_seqlens; a.scale = scale;
    a.N = cu_seqlens ? N : 0; a.B = B; a.T = T; a.H_q = H_q; a.H_kv = H_kv; a.D = D;
    const int rc = validate_attn(a);
    if (rc != KDA_OK) return rc;
    if (cu_seqlens && B != 1) return KDA_ERR_INVALID_ARG;
    if ((long long)B * T == 0) return nothing_to_do();
    return attend(a, own_ws, ws, ws_bytes, stream);
}

int paged(const kda_bf16_t *q, const kda_bf16_t *k_cache, const kda_bf16_t *v_cache, float scale,
          const int32_t *block_table, const int32_t *seq_lens, const int32_t *cu_seqlens, int N, int T, int H_q,
          int H_kv, int D, int num_blocks, int block_size, int max_blocks, kda_bf16_t *out, float *lse, bool own_ws,
          void *ws, size_t ws_bytes, cudaStream_t stream) {
    kda::AttnArgs a = {};
    a.q = q; a.k = k_cache; a.v = v_cache; a.out = out; a.lse = lse; a.cu = cu_seqlens; a.scale = scale;
    a.table = block_table; a.lens = seq_lens;
    a.N = N; a.B = 1; a.T = T; a.H_q = H_q; a.H_kv = H_kv; a.D = D;
    a.num_blocks = num_blocks; a.block_log2 = block_log2(block_size); a.max_blocks = max_blocks;
    if (a.block_log2 < 0) return KDA_ERR_UNSUPPORTED;
    const int rc = validate_attn(a);
    if (rc != KDA_OK) return rc;
    if (!cache_ok(num_blocks, a.block_log2) || (long long)num_blocks * H_kv > 0x7ffffffeLL || max_blocks < 0)
        return KDA_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return nothing_to_do();
    if ((!block_table && max_blocks > 0) || !seq_lens || !cu_seqlens || num_blocks == 0) return KDA_ERR_INVALID_ARG;
    return attend(a, own_ws, ws, ws_bytes, stream);
}
}  // namespace

extern "C" {

int kda_page_plan(const int32_t *cached_lens, const int32_t *new_lens, const int32_t *free_blocks,
                  const int32_t *free_start, int32_t *block_table, int N, int T, int max_blocks, int block_size,
                  int num_free, int32_t *cu_seqlens, int32_t *seq_lens, int32_t *slots, int32_t *positions,
                  int32_t *free_next, cudaStream_t stream) {
    const int lg = block_log2(block_size);
    if (lg < 0) return KDA_ERR_UNSUPPORTED;
    if (N < 0 || T < 0 || max_blocks < 0 || num_free < 0) return KDA_ERR_INVALID_ARG;
    if (!free_start || !free_next || !cu_seqlens) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!cached_lens || !new_lens || !seq_lens || (max_blocks > 0 && !block_table))) return KDA_ERR_INVALID_ARG;
    if ((T > 0 && (!slots || !positions)) || (num_free > 0 && !free_blocks)) return KDA_ERR_INVALID_ARG;
    if (!ints_aligned(cached_lens, new_lens, free_blocks, free_start, block_table, cu_seqlens, seq_lens, slots, positions,
                      free_next))
        return KDA_ERR_INVALID_ARG;
    kda::timing_begin(stream);
    return finish(kda::launch_page_plan(cached_lens, new_lens, free_blocks, free_start, block_table, N, T, max_blocks,
                                        lg, num_free, cu_seqlens, seq_lens, slots, positions, free_next, stream),
                  "page_plan_kernel", stream);
}

int kda_kv_write(const kda_bf16_t *k, const kda_bf16_t *v, const int32_t *slots, kda_bf16_t *k_cache,
                 kda_bf16_t *v_cache, int T, int H_kv, int D, int num_blocks, int block_size, cudaStream_t stream) {
    const int lg = block_log2(block_size);
    if (lg < 0 || (D != 64 && D != 128)) return KDA_ERR_UNSUPPORTED;
    if (T < 0 || H_kv <= 0 || !cache_ok(num_blocks, lg)) return KDA_ERR_INVALID_ARG;
    // 256 units of 16 bytes a thread block, and a 32-bit grid
    if ((long long)T * H_kv * (D / 8) > 0x7fffffffLL * 256) return KDA_ERR_INVALID_ARG;
    if (T == 0) return nothing_to_do();
    if (!k || !v || !slots || (num_blocks > 0 && (!k_cache || !v_cache))) return KDA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slots, 4))
        return KDA_ERR_INVALID_ARG;
    kda::timing_begin(stream);
    return finish(kda::launch_kv_write(k, v, slots, k_cache, v_cache, T, H_kv, D, num_blocks, lg, stream),
                  "kv_write_kernel", stream);
}

size_t kda_attn_workspace_size(int D) { return D == 64 || D == 128 ? kda::attn_workspace_bytes(D) : 0; }

int kda_attn_fwd(const kda_bf16_t *q, const kda_bf16_t *k, const kda_bf16_t *v, float scale,
                 const int32_t *cu_seqlens, int N, int B, int T, int H_q, int H_kv, int D, kda_bf16_t *out, float *lse,
                 cudaStream_t stream) {
    return prompt(q, k, v, scale, cu_seqlens, N, B, T, H_q, H_kv, D, out, lse, true, nullptr, 0, stream);
}

int kda_attn_fwd_ws(const kda_bf16_t *q, const kda_bf16_t *k, const kda_bf16_t *v, float scale,
                    const int32_t *cu_seqlens, int N, int B, int T, int H_q, int H_kv, int D, kda_bf16_t *out,
                    float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
    return prompt(q, k, v, scale, cu_seqlens, N, B, T, H_q, H_kv, D, out, lse, false, ws, ws_bytes, stream);
}

int kda_attn_paged(const kda_bf16_t *q, const kda_bf16_t *k_cache, const kda_bf16_t *v_cache, float scale,
                   const int32_t *block_table, const int32_t *seq_lens, const int32_t *cu_seqlens, int N, int T,
                   int H_q, int H_kv, int D, int num_blocks, int block_size, int max_blocks, kda_bf16_t *out,
                   float *lse, cudaStream_t stream) {
    return paged(q, k_cache, v_cache, scale, block_table, seq_lens, cu_seqlens, N, T, H_q, H_kv, D, num_blocks,
                 block_size, max_blocks, out, lse, true, nullptr, 0, stream);
}

int kda_attn_paged_ws(const kda_bf16_t *q, const kda_bf16_t *k_cache, const kda_bf16_t *v_cache, float scale,
                      const int32_t *block_table, const int32_t *seq_lens, const int32_t *cu_seqlens, int N, int T,
                      int H_q, int H_kv, int D, int num_blocks, int block_size, int max_blocks, kda_bf16_t *out,
                      float *lse, void *ws, size_t ws_bytes, cudaStream_t stream) {
    return paged(q, k_cache, v_cache, scale, block_table, seq_lens, cu_seqlens, N, T, H_q, H_kv, D, num_blocks,
                 block_size, max_blocks, out, lse, false, ws, ws_bytes, stream);
}

}  // extern "C"
