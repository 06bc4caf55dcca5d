// Lightning attention forward: linear attention with a fixed per-head decay,
// one fused chunked pass per (sequence, value head).
//
// Per sequence and value head h (state S in R^{V x K}, lambda = exp(-slope[h])):
//   S_t = lambda S_{t-1} + v_t k_t^T,        o_t = scale S_t q_t.
// Over a chunk of C = 64 rows starting from S_0, with Gam_r = -(r + 1) slope
// (in-chunk log decay up to and including row r) and len rows:
//   O[r] = scale [ exp(Gam_r) (S_0 q_r) + sum_{j<=r} P[r][j] v_j ],   P[r][j] = exp(Gam_r - Gam_j) q_r.k_j
//   S_C  = exp(Gam_len) S_0 + Z^T,   Z^T[v][k] = sum_r v_r[v] k_r[k] exp(Gam_len - Gam_r)
// Z does not depend on S_0, so the only serial step from chunk to chunk is
// S <- exp(Gam_len) S + Z^T, one FMA per state element.
//
// One CTA per (sequence, value head).  16 epilogue warps keep S (fp32) in
// registers, thread (v, column group) owning S[v][k] for 32 values of k, and
// keep a bf16 copy of S in tensor memory as the A operand of the output MMA.
// Two issuer threads (one lane of each of two more warps) drive the tensor
// core, since one thread issues at most one MMA every ~65 cycles: the state
// issuer streams q, k, v chunks with TMA (three stages, zero fill past the
// tensor) and issues A and M3; the output issuer issues M2 and M1:
//   A   Da   = Q K^T                  (M = 64,  N = 64, K = 128; A, B from shared memory)
//   M3  Z^T  = V^T (Kd_hi + Kd_lo)     (M = 128, N = 128, K = 64; V and Kd MN-major)
//   M2  Y2^T = V^T P^T                 (M = 128, N = 64,  K = 64)
//   M1  Y1^T = S Q^T                   (M = 128, N = 64,  K = 128; S from tensor memory)
// All bf16 with fp32 accumulation.  Once A has read a stage, the epilogue
// rewrites its K rows in place as Kd_hi = bf16(k exp(Gam_len - Gam_r)) and
// stores the remainder Kd_lo in a double buffer, so the state update keeps
// ~16 bits; S and P enter the output products rounded to bf16, like the output
// itself.  P carries the factor scale, and the output O = scale exp(Gam_r) Y1 + Y2
// is transposed through shared memory (double-buffered) and leaves by one TMA tensor
// store per full chunk (16-byte stores of the valid rows for a sequence's last,
// partial chunk, whose other rows belong to the next sequence).  Every
// wait is bounded; a timeout records KDA_ERR_DEVICE_TIMEOUT and all roles stop.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_common.cuh"
#include "kda_tma.cuh"

namespace kda {

cudaError_t launch_plan(const int32_t *cu, int N, int B, int T, SeqDesc *seqs, ChunkDesc *chunks, int *order,
                        int *hdr, long long max_chunks, cudaStream_t stream);
long long max_chunks_for(int N, int B, int T, bool varlen);

constexpr int LA_EPI_WARPS = 16;
constexpr int LA_EPI = LA_EPI_WARPS * 32;
constexpr int LA_THREADS = LA_EPI + 64;   // + two issuer warps
constexpr int LA_NST = 3;                 // load stages

// A stage holds one chunk: Q, K, V as 64 rows x 128 bf16, each as two 8 KiB
// 128-byte-swizzled atoms (channels 0..63, 64..127), the layout a TMA box of
// 64 x 64 elements writes.  Row-major [row][channel] in this layout is at once
// the K-major operand over channels and the MN-major operand over rows.
constexpr uint32_t LA_STAGE = 49152;
constexpr uint32_t LA_Q = 0, LA_K = 16384, LA_V = 32768;
constexpr uint32_t LA_PB = LA_NST * LA_STAGE;   // 2 x 8 KiB   P [r][j] bf16, K-major
constexpr uint32_t LA_KL = LA_PB + 16384;       // 2 x 16 KiB  Kd_lo (stage layout)
constexpr uint32_t LA_OS = LA_KL + 32768;       // 2 x 16 KiB  output staging, bf16 [64 r][128 v]
constexpr uint32_t LA_BAR = LA_OS + 32768;
constexpr uint32_t LA_SLOT = LA_BAR + 128;
constexpr uint32_t LA_FLAG = LA_BAR + 132;
constexpr uint32_t LA_BYTES = LA_BAR + 256 + 1024;   // + alignment slack
static_assert(LA_BYTES <= 232448, "lightning-attention shared memory exceeds 227 KiB");

// tensor memory columns
constexpr uint32_t LT_Z = 0, LT_SA = 128, LT_Y1 = 192, LT_Y2 = 320, LT_DA = 448;

enum { LB_LD0 = 0, LB_A = LA_NST, LB_M3, LB_M12_0, LB_M12_1, LB_E1R0, LB_E1R1, LB_SBR, LB_OUT0, LB_OUT1, LB_COUNT };
static_assert(8 * LB_COUNT <= 128, "barrier area");

struct LaParams {
    const SeqDesc *seqs;
    const int *order;
    const int *hdr;
    const float *slope;
    float scale;
    const float *init;
    float *fin;
    uint16_t *out;
    int H_qk, H_v, nseq;
};

__global__ __launch_bounds__(LA_THREADS, 1) void la_fwd_kernel(const __grid_constant__ CUtensorMap tq,
                                                               const __grid_constant__ CUtensorMap tk,
                                                               const __grid_constant__ CUtensorMap tv,
                                                               const __grid_constant__ CUtensorMap tout,
                                                               const LaParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    if (p.hdr[1] == 0) return;
    const int h = blockIdx.x % p.H_v, rank = blockIdx.x / p.H_v;
    if (rank >= p.nseq) return;
    const int seq = p.order[rank];
    const SeqDesc sd = p.seqs[seq];
    const int n = sd.nchunk, hq = h / (p.H_v / p.H_qk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(sm), bar = sbase + LA_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + LA_FLAG);

    if (tid == 0) {
        for (int i = 0; i < LB_E1R0; ++i) mbar_init(bar + 8 * i, 1);
        for (int i = LB_E1R0; i < LB_COUNT; ++i) mbar_init(bar + 8 * i, LA_EPI_WARPS);
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == 0) tmem_alloc(sbase + LA_SLOT, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + LA_SLOT);
    const float sl2 = p.slope[h] * LOG2E;   // decay per token, log2 units
    auto fail = [&]() {
        set_status(KDA_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp >= LA_EPI_WARPS) {
        // ------------------------------------------------------------ issuers (one lane each)
        const uint32_t id_a = idesc_bf16(64, 64);
        const uint32_t id_3 = idesc_bf16(128, 128) | (1u << 15) | (1u << 16);
        const uint32_t id_2 = idesc_bf16(128, 64) | (1u << 15);
        const uint32_t id_1 = idesc_bf16(128, 64);
        // descriptors of stage 0 / buffer 0; other operands add (byte offset >> 4) to the address field
        const uint64_t dQ = umma_desc(sbase + LA_Q, 16, 1024), dK = umma_desc(sbase + LA_K, 16, 1024);
        const uint64_t dKm = umma_desc(sbase + LA_K, 8192, 1024), dV = umma_desc(sbase + LA_V, 8192, 1024);
        const uint64_t dKL = umma_desc(sbase + LA_KL, 8192, 1024), dPB = umma_desc(sbase + LA_PB, 16, 1024);
        auto stg = [](int c) { return (uint64_t)((c % LA_NST) * (LA_STAGE >> 4)); };
        auto kmaj = [](int ks) { return (uint64_t)((((ks >> 2) * 8192) + (ks & 3) * 32) >> 4); };
        bool ok = true;
        if (lane == 0 && warp == LA_EPI_WARPS) {
            // ---- state issuer: loads, A (Da = Q K^T), M3 (Z^T = V^T Kd)
            auto load = [&](int c) {
                const int s = c % LA_NST;
                const uint32_t b = bar + 8 * (LB_LD0 + s), dst = sbase + s * LA_STAGE;
                const int row = sd.tok + c * CH;
                mbar_expect_tx(b, LA_STAGE);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    tma_load_3d(dst + LA_Q + half * 8192, &tq, 64 * half, hq, row, b);
                    tma_load_3d(dst + LA_K + half * 8192, &tk, 64 * half, hq, row, b);
                    tma_load_3d(dst + LA_V + half * 8192, &tv, 64 * half, h, row, b);
                }
            };
            auto mma_a = [&](int c) {
                const uint64_t o = stg(c);
#pragma unroll
                for (int ks = 0; ks < KD / 16; ++ks)
                    umma_bf16(tmem + LT_DA, dQ + o + kmaj(ks), dK + o + kmaj(ks), id_a, ks > 0 ? 1u : 0u);
                umma_commit(bar + 8 * LB_A);
            };
            for (int c = 0; c < n && c < LA_NST; ++c) load(c);
            if (n > 0) {
                if (!mbar_wait(bar + 8 * LB_LD0, 0)) ok = false;
                else {
                    tc_fence_after();
                    mma_a(0);
                }
            }
            for (int c = 0; ok && c < n && !*abort_flag; ++c) {
                const uint64_t o = stg(c);
                // E1 of chunk c is done: Da is free, so A of the next chunk goes first
                if (!mbar_wait(bar + 8 * (LB_E1R0 + (c & 1)), (c >> 1) & 1)) { ok = false; break; }
                if (c + 1 < n) {
                    if (!mbar_wait(bar + 8 * (LB_LD0 + (c + 1) % LA_NST), ((c + 1) / LA_NST) & 1)) { ok = false; break; }
                    tc_fence_after();
                    mma_a(c + 1);
                }
                // M3: Z was read by the previous state update (SBR #c)
                if (!mbar_wait(bar + 8 * LB_SBR, c & 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < CH / 16; ++ks)
                        umma_bf16(tmem + LT_Z, dV + o + ks * (2048 >> 4),
                                  (part ? dKL + (uint64_t)((c & 1) * (16384 >> 4)) : dKm + o) + ks * (2048 >> 4), id_3,
                                  (part > 0 || ks > 0) ? 1u : 0u);
                umma_commit(bar + 8 * LB_M3);
                // refill this stage once M3, M2 and M1 of chunk c have read it
                if (c + LA_NST < n) {
                    if (!mbar_wait(bar + 8 * LB_M3, c & 1) ||
                        !mbar_wait(bar + 8 * (LB_M12_0 + (c & 1)), (c >> 1) & 1)) { ok = false; break; }
                    load(c + LA_NST);
                }
            }
        } else if (lane == 0) {
            // ---- output issuer: M2 (Y2^T = V^T P^T), then M1 (Y1^T = S Q^T) once S of the previous chunk is
            //      in tensor memory
            for (int c = 0; ok && c < n && !*abort_flag; ++c) {
                const uint64_t o = stg(c);
                const int b = c & 1;
                if (!mbar_wait(bar + 8 * (LB_LD0 + c % LA_NST), (c / LA_NST) & 1) ||
                    !mbar_wait(bar + 8 * (LB_E1R0 + b), (c >> 1) & 1)) { ok = false; break; }
                if (c >= 2 && !mbar_wait(bar + 8 * (LB_OUT0 + b), ((c >> 1) - 1) & 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < CH / 16; ++ks)
                    umma_bf16(tmem + LT_Y2 + 64 * b, dV + o + ks * (2048 >> 4), dPB + (uint64_t)(b * (8192 >> 4) + ks * 2),
                              id_2, ks > 0 ? 1u : 0u);
                if (!mbar_wait(bar + 8 * LB_SBR, c & 1)) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < KD / 16; ++ks)
                    umma_bf16_ta(tmem + LT_Y1 + 64 * b, tmem + LT_SA + 8 * ks, dQ + o + kmaj(ks), id_1, ks > 0 ? 1u : 0u);
                umma_commit(bar + 8 * (LB_M12_0 + b));
            }
        }
        if (lane == 0) {
            if (!ok) fail();
            if (*abort_flag) {
                // let whatever is still in flight land before the CTA releases TMEM (bounded)
                for (int i = 0; i < LB_E1R0; ++i)
                    for (uint32_t pp = 0; pp < 2; ++pp) mbar_wait(bar + 8 * i, pp, 1u << 14);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q4 = warp & 3, cg = warp >> 2;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const int vme = q4 * 32 + lane;   // state row v (lane of the M = 128 accumulators)
        const int rme = q4 * 16 + lane;   // chunk row of the M = 64 accumulator Da (lanes < 16)
        float S[32];                      // S[vme][32 cg + j]
        const size_t st0 = (((size_t)seq * p.H_v + h) * KD + vme) * KD + 32 * cg;
        if (p.init) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(p.init + st0 + j);
                S[j] = x.x; S[j + 1] = x.y; S[j + 2] = x.z; S[j + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) S[j] = 0.f;
        }
        // bf16 S (columns 16 cg .. 16 cg + 15 of the A operand: k = 32 cg + 2 w, 2 w + 1) and release
        auto write_sa = [&]() {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(S[2 * i], S[2 * i + 1]);
            tmem_st16(tmem + LT_SA + lane_off + 16 * cg, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8 * LB_SBR);
        };
        write_sa();
        const float lam = ex2(-sl2);
        // row decays of this thread's two 16-byte units of K (rows tid / 16 and tid / 16 + 32) for a
        // full chunk: exp(Gam_63 - Gam_r)
        float edr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) edr[i] = ex2(-sl2 * (float)(CH - 1 - ((tid >> 4) + 32 * i)));
        const float eq0 = p.scale * ex2(-sl2 * (float)(16 * cg + 1));   // scale exp(Gam_r), first output row
        // P factors: below the diagonal block the walk starts at column e = 15 with scale lambda^(r - j)
        // (r - j >= 1); on it the factor only advances on kept columns (e <= lane), starting at scale
        const float pscale0 = p.scale * ex2(-sl2 * (float)max(rme - 16 * cg - 15, 0));
        const float pscale_diag = p.scale;

        // E1 of chunk c: P from Da; Kd = K exp(Gam_len - Gam_r) (hi in place, lo in its buffer).
        // P[c & 1] and Kd_lo[c & 1] were last read by M2 / M3 of chunk c - 2, which the state
        // update of chunk c - 2 waited for, earlier in program order.
        auto e1 = [&](int c) -> bool {
            const int s = c % LA_NST;
            unsigned char *stg = sm + s * LA_STAGE;
            const int len = min(CH, sd.len - c * CH);
            if (!mbar_wait_hint(bar + 8 * (LB_LD0 + s), (c / LA_NST) & 1) || !mbar_wait_hint(bar + 8 * LB_A, c & 1)) return false;
            tc_fence_after();
            {
                // P block (rows 16 q4 .., columns 16 cg ..) times scale: zero above the diagonal block;
                // below and on it scale lambda^(r - j), built from lambda^(r - 16 cg - 15) by factors of
                // lambda going down the columns, masked (j > r) on the diagonal block
                unsigned char *pb = sm + LA_PB + (c & 1) * 8192;
                float o[16];
                if (cg > q4) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                } else {
                    uint32_t x[16];
                    tmem_ld16_nowait(tmem + LT_DA + lane_off + 16 * cg, x);
                    float f = cg < q4 ? pscale0 : pscale_diag;
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 15; e >= 0; --e) {
                        o[e] = __uint_as_float(x[e]) * f;
                        if (cg < q4 || e <= lane) f *= lam;
                    }
                    if (cg == q4) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = e <= lane ? o[e] : 0.f;
                    }
                }
                if (lane < 16) {
#pragma unroll
                    for (int hlf = 0; hlf < 2; ++hlf)
                        *reinterpret_cast<uint4 *>(pb + sw128_off(rme, 32 * cg + 16 * hlf, CH)) =
                            make_uint4(pack_bf16x2(o[8 * hlf + 0], o[8 * hlf + 1]), pack_bf16x2(o[8 * hlf + 2], o[8 * hlf + 3]),
                                       pack_bf16x2(o[8 * hlf + 4], o[8 * hlf + 5]), pack_bf16x2(o[8 * hlf + 6], o[8 * hlf + 7]));
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (tid >> 4) + 32 * i, c16 = tid & 15;
                const uint32_t off = sw128_off(r, 16 * c16, CH);
                const float ed = len == CH ? edr[i] : (r < len ? ex2(-sl2 * (float)(len - 1 - r)) : 0.f);
                const uint4 kw = *reinterpret_cast<const uint4 *>(stg + LA_K + off);
                const uint32_t ka[4] = {kw.x, kw.y, kw.z, kw.w};
                uint32_t kh[4], kl[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // packed fp32 pairs: d = k ed, lo = d - bf16(d)
                    const float2 d = __fmul2_rn(make_float2(bf16_lo(ka[e]), bf16_hi(ka[e])), make_float2(ed, ed));
                    kh[e] = pack_bf16x2(d.x, d.y);
                    const float2 r = __ffma2_rn(make_float2(bf16_lo(kh[e]), bf16_hi(kh[e])), make_float2(-1.f, -1.f), d);
                    kl[e] = pack_bf16x2(r.x, r.y);
                }
                *reinterpret_cast<uint4 *>(stg + LA_K + off) = make_uint4(kh[0], kh[1], kh[2], kh[3]);
                *reinterpret_cast<uint4 *>(sm + LA_KL + (c & 1) * 16384 + off) = make_uint4(kl[0], kl[1], kl[2], kl[3]);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8 * (LB_E1R0 + (c & 1)));
            return true;
        };
        // E2 of chunk c: S <- exp(Gam_len) S + Z^T, then the bf16 copy for the next chunk's M1
        auto e2 = [&](int c) -> bool {
            const int len = min(CH, sd.len - c * CH);
            if (!mbar_wait_hint(bar + 8 * LB_M3, c & 1) || !mbar_wait_hint(bar + 8 * (LB_M12_0 + (c & 1)), (c >> 1) & 1))
                return false;
            tc_fence_after();
            const float g = ex2(-sl2 * (float)len);
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
                uint32_t z[16];
                tmem_ld16_nowait(tmem + LT_Z + lane_off + 32 * cg + 16 * hlf, z);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 r = __ffma2_rn(make_float2(S[16 * hlf + j], S[16 * hlf + j + 1]), make_float2(g, g),
                                                make_float2(__uint_as_float(z[j]), __uint_as_float(z[j + 1])));
                    S[16 * hlf + j] = r.x;
                    S[16 * hlf + j + 1] = r.y;
                }
            }
            write_sa();
            return true;
        };
        // output of chunk c: O[r][v] = scale (exp(Gam_r) Y1^T[v][r] + Y2^T[v][r]) for r = 16 cg .. 16 cg + 15,
        // through staging buffer c & 1: a full chunk leaves by one TMA store issued by thread 0, a
        // partial one by 16-byte stores of its valid rows.  Before the barrier thread 0 waits for
        // its previous store (chunk c - 1, the other buffer) to finish reading, so that after it
        // every thread may rewrite that buffer for chunk c + 1.
        auto emit = [&](int c) {
            const int b = c & 1, len = min(CH, sd.len - c * CH);
            uint16_t *os = reinterpret_cast<uint16_t *>(sm + LA_OS + b * 16384);
            float f = eq0;
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
                uint32_t y1[8], y2[8];
                tmem_ld8_nowait(tmem + LT_Y1 + 64 * b + lane_off + 16 * cg + 8 * hlf, y1);
                tmem_ld8_nowait(tmem + LT_Y2 + 64 * b + lane_off + 16 * cg + 8 * hlf, y2);
                tmem_wait_ld();
                if (hlf == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + 8 * (LB_OUT0 + b));
                }
                // rows 16 cg + 8 hlf + j take f = eq0 lambda^(8 hlf + j); row pairs walk by lambda^2
                float2 fp = make_float2(f, f * lam);
                const float2 l2 = make_float2(lam * lam, lam * lam);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 r = __ffma2_rn(fp, make_float2(__uint_as_float(y1[j]), __uint_as_float(y1[j + 1])),
                                                make_float2(__uint_as_float(y2[j]), __uint_as_float(y2[j + 1])));
                    os[(16 * cg + 8 * hlf + j) * KD + vme] = f_to_bf16(r.x);
                    os[(16 * cg + 8 * hlf + j + 1) * KD + vme] = f_to_bf16(r.y);
                    fp = __fmul2_rn(fp, l2);
                }
                f = fp.x;
            }
            fence_async_smem();
            if (tid == 0) bulk_wait_read_all();
            named_bar(1, LA_EPI);
            if (len == CH) {
                if (tid == 0) {
                    tma_store_3d(&tout, 0, h, sd.tok + c * CH, sbase + LA_OS + b * 16384);
                    bulk_commit();
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int u = tid + LA_EPI * i, r = u >> 4, c16 = u & 15;
                    if (r < len)
                        *reinterpret_cast<uint4 *>(p.out + ((size_t)(sd.tok + c * CH + r) * p.H_v + h) * KD + 8 * c16) =
                            *reinterpret_cast<const uint4 *>(os + r * KD + 8 * c16);
                }
            }
        };
        bool ok = n == 0 || e1(0);
        for (int c = 0; ok && c < n; ++c) {
            if (*abort_flag) { ok = false; break; }
            if (c + 1 < n && !e1(c + 1)) { ok = false; break; }
            if (!e2(c)) { ok = false; break; }
            emit(c);
        }
        if (!ok) fail();
        if (tid == 0) bulk_wait_all();   // the last output stores are done with shared memory
        if (ok && p.fin) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4 *>(p.fin + st0 + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side
namespace {
// [rows][heads][128] bf16, boxes of 64 channels x 1 head x 64 rows, 128-byte swizzle
cudaError_t make_map(CUtensorMap *m, const void *base, long long rows, int heads) {
    return tma_map_rows_heads(m, base, rows, heads, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t align256_la(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

// Plan tables only: header, sequence table, chunk table, order.
size_t la_workspace_bytes(int N, int B, int T, bool varlen) {
    const long long nseq = varlen ? N : B;
    const long long nck = max_chunks_for(N, B, T, varlen);
    size_t off = align256_la(256);
    off = align256_la(off + sizeof(SeqDesc) * (size_t)(nseq > 0 ? nseq : 1));
    off = align256_la(off + sizeof(ChunkDesc) * (size_t)(nck > 0 ? nck : 1));
    off = align256_la(off + sizeof(int) * (size_t)(nseq > 0 ? nseq : 1));
    return off;
}

cudaError_t launch_la_fwd(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *slope, float scale,
                          const float *init, float *fin, const int32_t *cu, int N, int B, int T, int H_qk, int H_v,
                          uint16_t *out, void *ws_ptr, cudaStream_t stream, int *launches) {
    const bool varlen = cu != nullptr;
    const int nseq = varlen ? N : B;
    const long long nck = max_chunks_for(N, B, T, varlen);
    char *base = static_cast<char *>(ws_ptr);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = base + off;
        off = align256_la(off + bytes);
        return p;
    };
    int *hdr = reinterpret_cast<int *>(take(256));
    SeqDesc *seqs = reinterpret_cast<SeqDesc *>(take(sizeof(SeqDesc) * (size_t)(nseq > 0 ? nseq : 1)));
    ChunkDesc *chunks = reinterpret_cast<ChunkDesc *>(take(sizeof(ChunkDesc) * (size_t)(nck > 0 ? nck : 1)));
    int *order = reinterpret_cast<int *>(take(sizeof(int) * (size_t)(nseq > 0 ? nseq : 1)));
    *launches = 0;
    cudaError_t e = launch_plan(cu, N, B, T, seqs, chunks, order, hdr, nck, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (nseq == 0) return cudaSuccess;
    const long long rows = (long long)B * T;
    CUtensorMap mq, mk, mv, mo;
    // a map needs at least one row; with no tokens the kernel only copies the states
    const void *qb = rows > 0 ? (const void *)q : (const void *)hdr;
    const void *kb = rows > 0 ? (const void *)k : (const void *)hdr;
    const void *vb = rows > 0 ? (const void *)v : (const void *)hdr;
    const void *ob = rows > 0 ? (const void *)out : (const void *)hdr;
    const long long r = rows > 0 ? rows : 1;
    if ((e = make_map(&mq, qb, r, rows > 0 ? H_qk : 1)) != cudaSuccess) return e;
    if ((e = make_map(&mk, kb, r, rows > 0 ? H_qk : 1)) != cudaSuccess) return e;
    if ((e = make_map(&mv, vb, r, rows > 0 ? H_v : 1)) != cudaSuccess) return e;
    // the output: whole 256-byte rows, no swizzle (the staging buffer is row-major [64 r][128 v])
    if ((e = tma_map_rows_heads(&mo, ob, r, rows > 0 ? H_v : 1, 128, CU_TENSOR_MAP_SWIZZLE_NONE)) != cudaSuccess)
        return e;
    if ((e = cudaFuncSetAttribute(la_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LA_BYTES)) !=
        cudaSuccess)
        return e;
    LaParams lp;
    lp.seqs = seqs; lp.order = order; lp.hdr = hdr; lp.slope = slope; lp.scale = scale;
    lp.init = init; lp.fin = fin; lp.out = out; lp.H_qk = H_qk; lp.H_v = H_v; lp.nseq = nseq;
    la_fwd_kernel<<<(unsigned)((long long)nseq * H_v), LA_THREADS, LA_BYTES, stream>>>(mq, mk, mv, mo, lp);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace kda
