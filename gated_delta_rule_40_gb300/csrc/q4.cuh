// The 4-bit cache format.
//
// 32 channels of a key or value share a scale byte b, which stands for s = 2^((b >> 3) - 15) (1 + (b & 7) / 8); a
// channel is a code c of 4 bits for the value (c - 8) s, c from 1 to 15.  Both factors have four significant bits
// or fewer, so every value is a bf16 number: attention's tensor-core operands are the values themselves.  (A block
// of 32 with a scale of 8 bits: 4.25 bits a channel.  Normal values keep 0.103 of their deviation as error.)
//
// The word of 8 channels holds channel 2j in bits 4j and channel 2j + 1 in bits 16 + 4j, so that one shift and one
// mask give a pair of neighbours in the two halves of a register.  A (block, kv head) is its rows' D / 2 code bytes,
// row after row, then their D / 32 scale bytes.
#pragma once

#include "kda_common.cuh"

namespace kda {

__host__ __device__ constexpr int q4_code_bytes(int D) { return D / 2; }
__host__ __device__ constexpr int q4_scale_bytes(int D) { return D / 32; }
__host__ __device__ constexpr int q4_row_bytes(int D) { return D / 2 + D / 32; }

// The scale that byte b stands for
__device__ __forceinline__ float q4_scale(uint32_t b) { return __uint_as_float((b + (112u << 3)) << 20); }

// The smallest scale byte whose sevenfold reaches `most` (finite or infinite), or the largest there is.  The product
// with 1/7 may fall below a scale that is exact, never above one that is not: those are 2^-4 apart.
__device__ __forceinline__ uint32_t q4_scale_byte(float most) {
    const int near = (int)(__float_as_uint(most * (1.f / 7.f)) >> 20) - (112 << 3);
    const uint32_t b = (uint32_t)min(max(near, 0), 255);
    return b < 255 && 7.f * q4_scale(b) < most ? b + 1 : b;
}

// Codes under a scale s are 8 + n, n nearest to x / s, halves away from zero.  Halves are numbers of 8 significant bits
// like bf16's x, so x / s is one exactly or is 2^-9 (of it) or more away: times 1 / s and 1 + 2^-12, both roundings
// included, a half rounds away from zero and nothing else crosses one.
__device__ __forceinline__ float q4_inverse(float s) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return y * (1.f + 0x1p-12f);
}

// (x s + d) for bf16 pairs, with one rounding
__device__ __forceinline__ uint32_t q4_fma(uint32_t x, uint32_t s, uint32_t d) {
    uint32_t y;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(s), "r"(d));
    return y;
}

// Values as bf16 pairs, 2^-23 of what they are, from codes in place.  Bits 0 .. 7 of a bf16 number alone are an integer
// times 2^-133, below the normal numbers and among the first of them alike: pair j of a word (channels 2j, 2j + 1) is
// 2^-133 c from bits 0 .. 3 or 2^-129 c from bits 4 .. 7, times 2^110 s or 2^106 s less 8 2^-23 s, all without a rounding.
// Nothing larger than 2^110 will do, as 2^110 times the largest s is near the largest number there is.
constexpr float Q4_UP = 8388608.f, Q4_LOG_UP = 23.f;
struct Q4Scale {
    uint32_t even, odd, off;
};
// ... of scale bytes in bytes 0 and 2 of `two`; two4 is 16, from memory: a product for the multiplier, which has room, not
// a shift
__device__ __forceinline__ Q4Scale q4_scales(uint32_t two, uint32_t two4) {
    return {two * two4 + 0x6f006f00u, two * two4 + 0x6d006d00u, two * two4 + 0xae00ae00u};
}
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int j, const Q4Scale &s) {
    return q4_fma((j < 2 ? word : word >> 8) & (j & 1 ? 0x00f000f0u : 0x000f000fu), j & 1 ? s.odd : s.even, s.off);
}

}  // namespace kda
