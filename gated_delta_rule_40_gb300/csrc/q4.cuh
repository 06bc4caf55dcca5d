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

// Pair j (channels 2j, 2j + 1) of a word as bf16 16 + c: the code below the leading bit of 16's mantissa
__device__ __forceinline__ uint32_t q4_raw(uint32_t word, int j) {
    const uint32_t x = j == 0 ? word << 3 : word >> (4 * j - 3);
    return (x & 0x00780078u) | 0x41804180u;
}
// (x & mask) | bit in one instruction: with a mask and a bit that the compiler knows it makes two, so they are arguments
// of the kernels
__device__ __forceinline__ uint32_t q4_masked(uint32_t x, uint32_t mask, uint32_t bit) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;\n" : "=r"(y) : "r"(x), "r"(mask), "r"(bit));
    return y;
}
// (raw - 24) s with one rounding, which there is none of: s and 24 s as bf16 pairs, both exact
__device__ __forceinline__ uint32_t q4_value(uint32_t raw, uint32_t s2, uint32_t minus24s2) {
    uint32_t y;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(raw), "r"(s2), "r"(minus24s2));
    return y;
}
// Scale bytes b (in byte 0 and byte 2 of `two`, the others ignored) as a bf16 pair, and -24 times it
__device__ __forceinline__ uint32_t q4_scale2(uint32_t two) { return (two & 0x00ff00ffu) * 16u + 0x38003800u; }
__device__ __forceinline__ uint32_t q4_offset2(uint32_t s2) {
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(s2), "r"(0xc1c0c1c0u));   // -24
    return y;
}

}  // namespace kda
