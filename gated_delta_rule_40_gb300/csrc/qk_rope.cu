// Norms of queries and keys for each head with the position rotation in the same pass, and their gradients.
//
// With r = 1 / sqrt(mean x^2 + eps), y = x r w, and the pair (y_a, y_b) of frequency f turned by the angle
// position x f.  Backward, with g the gradient turned back: dw = sum g x r over tokens and heads,
// dx = r (g w - x r mean(g w x r)).
//
// Angle.  position x f in fp32 is off by radians at far positions, so angles are kept in turns as fixed-point
// fractions of 64 bits: F = f / (2 pi) 2^64 from f's mantissa times 128 bits of 1 / (2 pi) (Payne and Hanek's
// reduction), position x F modulo 2^64 is the fraction of a turn to 2^-33 at any int32 position.  It is rounded to fp32,
// by 2^-26 of a turn at most, which moves a cosine by 2^-23, and the function of pi x takes it from there.
//
// Layout.  A row (a head's D channels) is D / 8 lanes with two runs of four channels each: a lane that turns
// holds both channels of its four pairs (half-split pairs: 4l .. and R / 2 + 4l ..; neighbours: 8l ..), so a
// rotation needs no exchange between lanes.  A warp takes 2 (D = 128) or 4 rows at a time of one token, whose
// four frequencies a lane its rows compute together once, and has four such groups' loads in flight, at
// addresses that are one and constants.  Warps walk the tokens; where there are few, a token's rows are
// shared out among several.
//
// What bounds it, and what it measured on the GPU: DRAM.  32768 tokens x 40 heads of 128 in 107 us, 6.3 TB/s (0.93 of
// a copy; a warp a token 112 us, with an address for each row 122 us); gradients of 16384 tokens, which leave as
// fp32, in 104 us and 2 us for the weights' sum, 6.4 TB/s.  Packed fp32 pairs took 146 us: pairs of registers for
// them cost more moves than they save.  A call of 64 tokens takes 3.1 us, and the host 17.
#include "qk_rope.h"
#include "kda_common.cuh"
#include "launch.h"

#include <type_traits>

namespace kda {
namespace {

constexpr int QR_THREADS = 256, QR_WARPS = QR_THREADS / 32;
constexpr int QR_FWD_CTAS = 3, QR_BWD_CTAS = 2;   // of an SM at once, by registers

// 1 / (2 pi), the first 128 bits after the binary point
constexpr unsigned long long INV_2PI_HI = 0x28be60db9391054aull, INV_2PI_LO = 0x7f09d5f47d4d3770ull;

// f / (2 pi) as a fraction of a turn, modulo 1, in units of 2^-64; |f| < 2^24
__device__ unsigned long long turns_of(float f) {
    const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255u;
    const unsigned long long m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
    const int s = 150 - (int)(e ? e : 1u);   // f = m 2^-s
    const unsigned long long c = __umul64hi(m, INV_2PI_LO), lo = m * INV_2PI_HI, p1 = lo + c;
    const unsigned long long p2 = __umul64hi(m, INV_2PI_HI) + (p1 < lo ? 1 : 0);
    const unsigned long long t = s >= 128 ? 0 : s >= 64 ? p2 >> (s - 64) : s > 0 ? (p1 >> s) | (p2 << (64 - s)) : p1;
    return (u >> 31) ? 0 - t : t;
}

struct Lane {
    int at[2];   // first channels of the two runs
    bool turns;
};
template <int D>
__device__ __forceinline__ Lane lane_of(const QkRopeArgs &p, int l) {
    Lane x;
    const int turning = p.rot / 8;   // lanes of a row that turn
    x.turns = l < turning;
    if (!p.interleaved && x.turns) {
        x.at[0] = 4 * l;
        x.at[1] = p.rot / 2 + 4 * l;
    } else {   // neighbouring pairs, and the channels behind the turned ones
        x.at[0] = 8 * l;
        x.at[1] = 8 * l + 4;
    }
    return x;
}

// cos and sin of a lane's four frequencies at the token's position; the rows of a warp share the work
template <int D>
__device__ __forceinline__ void angles(const QkRopeArgs &p, const unsigned long long *turns, const bool *wild, int pos,
                                       int lane, bool on, float (&c)[4], float (&s)[4]) {
    constexpr int L = D / 8, ROWS = 32 / L, EACH = 4 / ROWS;
    const int row = lane / L;
    float mc[EACH], ms[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const long long t = (long long)((unsigned long long)pos * turns[j]);   // in [-1/2, 1/2) of a turn
        float sn, cs;
        sincospif((float)t * 0x1p-63f, &sn, &cs);
        mc[j] = !on ? 1.f : wild[j] ? NAN : cs;
        ms[j] = !on ? 0.f : wild[j] ? NAN : sn;
    }
    const int l = lane - row * L;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        c[j] = __shfl_sync(0xffffffffu, mc[j % EACH], (j / EACH) * L + l);
        s[j] = __shfl_sync(0xffffffffu, ms[j % EACH], (j / EACH) * L + l);
    }
}

// This lane's share of the frequencies (of its row's place in the warp)
template <int D>
__device__ __forceinline__ void load_turns(const QkRopeArgs &p, int lane, bool on, unsigned long long *turns, bool *wild) {
    constexpr int L = D / 8, ROWS = 32 / L, EACH = 4 / ROWS;
    const int row = lane / L, l = lane - row * L;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        const float f = on ? p.freqs[4 * l + row * EACH + j] : 0.f;
        wild[j] = !(fabsf(f) < 0x1p24f);
        turns[j] = turns_of(f);
    }
}

// Turns the pairs of x by the angles (c, s)
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[4], const float (&s)[4], bool interleaved, bool on) {
    if (!on) return;
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * c[j] - b * s[j];
            x[2 * j + 1] = a * s[j] + b * c[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[j], b = x[4 + j];
            x[j] = a * c[j] - b * s[j];
            x[4 + j] = a * s[j] + b * c[j];
        }
    }
}

__device__ __forceinline__ void unpack(const uint2 &u, float *x) {
    x[0] = bf16_lo(u.x);
    x[1] = bf16_hi(u.x);
    x[2] = bf16_lo(u.y);
    x[3] = bf16_hi(u.y);
}

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Loads the weights of a lane's channels
__device__ __forceinline__ void load_weight(const float *w, const Lane &x, float (&out)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = w ? w[x.at[j >> 2] + (j & 3)] : 1.f;
}

}  // namespace

// ---------------------------------------------------------------- forward
template <int D, bool NORM, bool PAIRS>
__global__ __launch_bounds__(QR_THREADS, QR_FWD_CTAS) void qk_rope_kernel(const QkRopeArgs p, int per, int chunks) {
    constexpr int L = D / 8, ROWS = 32 / L, EACH = 4 / ROWS, UNROLL = 4;
    const int lane = threadIdx.x & 31, row = lane / L, l = lane - row * L;
    const Lane x = lane_of<D>(p, l);
    unsigned long long turns[EACH];
    bool wild[EACH];
    load_turns<D>(p, lane, x.turns, turns, wild);
    const long long items = (long long)p.T * chunks;
    for (long long item = (long long)blockIdx.x * QR_WARPS + (threadIdx.x >> 5); item < items;
         item += (long long)gridDim.x * QR_WARPS) {
        const long long t = item / chunks;
        const int pos = p.positions[t];
        if (pos < 0) continue;   // a padded token
        float c[4], s[4];
        angles<D>(p, turns, wild, pos, lane, x.turns, c, s);
        const int gq = (p.H_q + ROWS - 1) / ROWS, gk = (p.H_kv + ROWS - 1) / ROWS;
        const int g0 = (int)(item - t * chunks) * per, g1 = min(g0 + per, gq + gk);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const int from = part ? max(g0, gq) : g0, to = part ? g1 : min(g1, gq), base = part ? gq : 0;
            if (from >= to) continue;
            const int heads = part ? p.H_kv : p.H_q, h0 = (from - base) * ROWS + row;
            const uint16_t *in = (part ? p.k + t * p.k_stride : p.q + t * p.q_stride) + h0 * D;
            uint16_t *out = (part ? p.k_out : p.q_out) + (t * heads + h0) * D;
            float w[8];
            if (NORM) load_weight(part ? p.k_weight : p.q_weight, x, w);
            // UNROLL rows, all of which there are where ALL is true; addresses are the first's and constants
            auto rows = [&](auto all, int left) {   // left: heads from the first row's on
                constexpr bool ALL = decltype(all)::value;
                uint2 u[UNROLL][2];
#pragma unroll
                for (int i = 0; i < UNROLL; ++i)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        u[i][b] = ALL || i * ROWS < left ? *reinterpret_cast<const uint2 *>(in + x.at[b] + i * ROWS * D) : make_uint2(0, 0);
#pragma unroll
                for (int i = 0; i < UNROLL; ++i) {
                    float v[8];
                    unpack(u[i][0], v);
                    unpack(u[i][1], v + 4);
                    if (NORM) {
                        float sum = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum += v[j] * v[j];
                        const float r = rsqrtf(row_sum<L>(sum) * (1.f / D) + p.eps);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = v[j] * r * w[j];
                    }
                    turn(v, c, s, PAIRS, x.turns);
                    if (ALL || i * ROWS < left) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            *reinterpret_cast<uint2 *>(out + x.at[b] + i * ROWS * D) =
                                make_uint2(pack_bf16x2(v[4 * b], v[4 * b + 1]), pack_bf16x2(v[4 * b + 2], v[4 * b + 3]));
                    }
                }
            };
            const int end = min((to - base) * ROWS, heads);   // of this warp's heads
            for (int g = from; g < to; g += UNROLL) {
                const int first = (g - base) * ROWS;
                if (first + UNROLL * ROWS <= end) rows(std::true_type{}, 0);
                else rows(std::false_type{}, end - first - row);
                in += UNROLL * ROWS * D;
                out += UNROLL * ROWS * D;
            }
        }
    }
}

// ---------------------------------------------------------------- backward
// Each warp walks tokens with a fixed stride and keeps the weights' gradients of its rows in registers; a CTA
// adds its warps' up in a fixed order, and qk_rope_dw_kernel the CTAs', so that bits repeat.
template <int D, bool NORM, bool PAIRS>
__global__ __launch_bounds__(QR_THREADS, QR_BWD_CTAS) void qk_rope_bwd_kernel(const QkRopeArgs p, int per, int chunks, float *partial) {
    constexpr int L = D / 8, ROWS = 32 / L, EACH = 4 / ROWS, UNROLL = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane / L, l = lane - row * L;
    grid_dep_launch();   // the sum of the weights' gradients may come as soon as CTAs leave
    const Lane x = lane_of<D>(p, l);
    unsigned long long turns[EACH];
    bool wild[EACH];
    load_turns<D>(p, lane, x.turns, turns, wild);
    const int gq = (p.H_q + ROWS - 1) / ROWS, gk = (p.H_kv + ROWS - 1) / ROWS;
    float dw[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.f;
    const long long items = (long long)p.T * chunks;
    for (long long item = (long long)blockIdx.x * QR_WARPS + warp; item < items; item += (long long)gridDim.x * QR_WARPS) {
        const long long t = item / chunks;
        const int pos = p.positions[t];
        if (pos < 0) continue;
        float c[4], s[4];
        angles<D>(p, turns, wild, pos, lane, x.turns, c, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = -s[j];
        const int g0 = (int)(item - t * chunks) * per, g1 = min(g0 + per, gq + gk);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int from = part ? max(g0, gq) : g0, to = part ? g1 : min(g1, gq), base = part ? gq : 0;
            if (from >= to) continue;
            const int heads = part ? p.H_kv : p.H_q, h0 = (from - base) * ROWS + row;
            const uint16_t *in = (part ? p.k + t * p.k_stride : p.q + t * p.q_stride) + h0 * D;
            const uint16_t *dy = (part ? p.dk_out : p.dq_out) + (t * heads + h0) * D;
            float *out = (part ? p.dk : p.dq) + (t * heads + h0) * D;
            float w[8];
            if (NORM) load_weight(part ? p.k_weight : p.q_weight, x, w);
            // as in the forward
            auto rows = [&](auto all, int left) {
                constexpr bool ALL = decltype(all)::value;
                uint2 u[UNROLL][2], d[UNROLL][2];
#pragma unroll
                for (int i = 0; i < UNROLL; ++i)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const bool on = ALL || i * ROWS < left;
                        d[i][b] = on ? *reinterpret_cast<const uint2 *>(dy + x.at[b] + i * ROWS * D) : make_uint2(0, 0);
                        if (NORM) u[i][b] = on ? *reinterpret_cast<const uint2 *>(in + x.at[b] + i * ROWS * D) : make_uint2(0, 0);
                    }
#pragma unroll
                for (int i = 0; i < UNROLL; ++i) {
                    float v[8];
                    unpack(d[i][0], v);
                    unpack(d[i][1], v + 4);
                    turn(v, c, s, PAIRS, x.turns);
                    if (NORM) {
                        float y[8], sum = 0.f, dot = 0.f;
                        unpack(u[i][0], y);
                        unpack(u[i][1], y + 4);
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum += y[j] * y[j];
                        const float r = rsqrtf(row_sum<L>(sum) * (1.f / D) + p.eps);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            y[j] *= r;
                            if (ALL || i * ROWS < left) dw[part][j] += v[j] * y[j];
                            v[j] *= w[j];
                            dot += v[j] * y[j];
                        }
                        dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = r * (v[j] - y[j] * dot);
                    }
                    if (ALL || i * ROWS < left) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            *reinterpret_cast<float4 *>(out + x.at[b] + i * ROWS * D) =
                                make_float4(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]);
                    }
                }
            };
            const int end = min((to - base) * ROWS, heads);
            for (int g = from; g < to; g += UNROLL) {
                const int first = (g - base) * ROWS;
                if (first + UNROLL * ROWS <= end) rows(std::true_type{}, 0);
                else rows(std::false_type{}, end - first - row);
                in += UNROLL * ROWS * D;
                dy += UNROLL * ROWS * D;
                out += UNROLL * ROWS * D;
            }
        }
    }
    if constexpr (NORM) {
        if (!partial) return;
        __shared__ float s_dw[QR_WARPS][2][D];
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = dw[part][j];   // the warp's rows
#pragma unroll
                for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (row == 0) s_dw[warp][part][x.at[j >> 2] + (j & 3)] = v;
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += QR_THREADS) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < QR_WARPS; ++k) v += s_dw[k][i / D][i % D];
            partial[(size_t)blockIdx.x * 2 * D + i] = v;
        }
    }
}

// Sum of the CTAs' gradients of both weights: 8 columns a CTA, 32 rows of partial sums at a time
__global__ __launch_bounds__(256) void qk_rope_dw_kernel(const float *partial, int n, int D, float *dwq, float *dwk) {
    __shared__ float s[32][8];
    const int col = blockIdx.x * 8 + (threadIdx.x & 7), r = threadIdx.x >> 3;
    float v = 0.f;
    grid_dep_wait();
    for (int i = r; i < n; i += 32) v += partial[(size_t)i * 2 * D + col];
    s[r][threadIdx.x & 7] = v;
    __syncthreads();
    if (r == 0) {
        v = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) v += s[k][threadIdx.x];
        float *out = col < D ? dwq : dwk;
        if (out) out[col < D ? col : col - D] = v;
    }
}

namespace {
constexpr int QR_MAX_CHUNKS = 32;   // looked at
constexpr int QR_ITEM_COST = 8, QR_LEAST = 4;

// Row groups a warp takes of a token, and the number of warps that its groups are shared out among: what makes the
// warps' rounds, each of which costs an item's start and angles (QR_ITEM_COST groups; 2 to 16 do as well) beside its
// groups, shortest for `warps` resident ones.  Fewer groups than QR_LEAST, those in flight together, make no round
// shorter: 64 tokens x 40 heads in 3.1 us with 4, 3.6 with 1 and 4.0 with 8, 150 tokens in 3.4, 4.4 and 4.3 us; 4096
// tokens in 16.1 us, with all groups of a token in one warp 19.9 us.
void split(const QkRopeArgs &a, int warps, int *per, int *chunks) {
    const int rows = a.D == 128 ? 2 : 4;
    const int groups = (a.H_q + rows - 1) / rows + (a.H_kv + rows - 1) / rows;
    *per = groups;
    *chunks = 1;
    long long best = ((long long)a.T + warps - 1) / warps * (max(groups, QR_LEAST) + QR_ITEM_COST);
    for (int c = 2; c <= groups && c <= QR_MAX_CHUNKS; ++c) {
        const int each = (groups + c - 1) / c;
        const long long cost = ((long long)a.T * c + warps - 1) / warps * (max(each, QR_LEAST) + QR_ITEM_COST);
        if (cost >= best) continue;
        best = cost;
        *per = each;
        *chunks = (groups + each - 1) / each;
    }
}

template <int D, bool NORM, bool PAIRS>
cudaError_t forward(const QkRopeArgs &a, cudaStream_t stream) {
    const int resident = sm_count() * QR_FWD_CTAS;
    if (resident == 0) return cudaErrorInvalidDevice;
    int per, chunks;
    split(a, resident * QR_WARPS, &per, &chunks);
    const long long want = ((long long)a.T * chunks + QR_WARPS - 1) / QR_WARPS, grid = want < resident ? want : resident;
    qk_rope_kernel<D, NORM, PAIRS><<<(unsigned)grid, QR_THREADS, 0, stream>>>(a, per, chunks);
    return cudaGetLastError();
}

template <int D, bool NORM, bool PAIRS>
cudaError_t backward(const QkRopeArgs &a, float *partial, int *n, cudaStream_t stream) {
    const int resident = sm_count() * QR_BWD_CTAS;
    if (resident == 0) return cudaErrorInvalidDevice;
    int per, chunks;
    split(a, resident * QR_WARPS, &per, &chunks);
    const long long want = ((long long)a.T * chunks + QR_WARPS - 1) / QR_WARPS;
    *n = (int)(want < resident ? want : resident);
    qk_rope_bwd_kernel<D, NORM, PAIRS><<<(unsigned)*n, QR_THREADS, 0, stream>>>(a, per, chunks, partial);
    return cudaGetLastError();
}

template <int D>
cudaError_t dispatch(const QkRopeArgs &a, bool bwd, float *partial, int *n, cudaStream_t s) {
    if (!bwd) {
        if (a.norm) return a.interleaved ? forward<D, true, true>(a, s) : forward<D, true, false>(a, s);
        return a.interleaved ? forward<D, false, true>(a, s) : forward<D, false, false>(a, s);
    }
    if (a.norm) return a.interleaved ? backward<D, true, true>(a, partial, n, s) : backward<D, true, false>(a, partial, n, s);
    return a.interleaved ? backward<D, false, true>(a, partial, n, s) : backward<D, false, false>(a, partial, n, s);
}
}  // namespace

size_t qk_rope_bwd_workspace_bytes(int D) { return sizeof(float) * 2 * D * MAX_SMS * QR_BWD_CTAS; }

cudaError_t launch_qk_rope(const QkRopeArgs &a, cudaStream_t stream) {
    return a.D == 64 ? dispatch<64>(a, false, nullptr, nullptr, stream) : dispatch<128>(a, false, nullptr, nullptr, stream);
}

cudaError_t launch_qk_rope_bwd(const QkRopeArgs &a, void *ws, cudaStream_t stream, int *launches) {
    const bool weights = a.norm && (a.dq_weight || a.dk_weight);
    float *partial = weights ? static_cast<float *>(ws) : nullptr;
    int n = 0;
    if (a.T > 0) {
        const cudaError_t e = a.D == 64 ? dispatch<64>(a, true, partial, &n, stream) : dispatch<128>(a, true, partial, &n, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (!weights) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * a.D / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = n > 0 ? 1 : 0;
    ++*launches;
    return cudaLaunchKernelEx(&cfg, qk_rope_dw_kernel, (const float *)partial, n, a.D, a.dq_weight, a.dk_weight);
}

}  // namespace kda
