// attend_convert.cuh -- what the matrix kernels of dspark_cache_attend share: codes to fp16, scaling of q's
// rows, constants of the weights.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dspark {

constexpr float kShift = 10.f;   // weights are 2^(t - m + kShift) <= 2^15
constexpr float kSlack = 5.f;    // m is raised when a score passes it by this

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// (w & mask) | or_bits in one instruction; or_bits in a register
template <uint32_t kMask>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t or_bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(kMask), "r"(or_bits));
    return r;
}

// Codes to fp16 by the old way of turning small integers into floating point: or them into the lowest bits of a power of
// two whose last place is 1, and subtract it. fp16 has that at 1024, and a code 4 bits up in the word counts 16 there:
//   (1024 + u) - (1024 + 8) = u - 8,   (1024 + 16 u) / 16 - (64 + 8) = u - 8,   exactly.
// The constants, kept in registers for a whole item: 1024 in both halves, 1032, 1/16, -72.
struct DequantConst {
    uint32_t magic, off, sixteenth, m72;
};

__device__ __forceinline__ DequantConst dequant_const()
{
    DequantConst c;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(c.magic));
    asm volatile("mov.b32 %0, 0x64086408;" : "=r"(c.off));
    asm volatile("mov.b32 %0, 0x2C002C00;" : "=r"(c.sixteenth));
    asm volatile("mov.b32 %0, 0xD480D480;" : "=r"(c.m72));
    return c;
}

// The 8 codes of a word times the scale pair s: h[j] = nibbles j and j + 4. 0x6400 | u is 1024 + u in fp16
// and 0x6400 | 16 u is 1024 + 16 u; the differences and products are exact.
__device__ __forceinline__ void dequant(uint32_t w, __half2 s, const DequantConst& c, uint32_t (&h)[4])
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t lo = and_or<0x000F000Fu>(w, c.magic), hi = and_or<0x00F000F0u>(w, c.magic);
        h[2 * k] = as_u32(__hmul2(__hsub2(as_half2(lo), as_half2(c.off)), s));
        h[2 * k + 1] = as_u32(__hmul2(__hfma2(as_half2(hi), as_half2(c.sixteenth), as_half2(c.m72)), s));
        w >>= 8;
    }
}

__device__ __forceinline__ uint32_t pack(float a, float b) { return as_u32(__floats2half2_rn(a, b)); }

// The power of two that takes a row of q whose largest magnitude has the exponent bits `ex` to 2^12 .. 2^13, and
// what its scores take back to log2 units with. Never 0: 0 times a masked score would be NaN.
__device__ __forceinline__ float row_up(int ex) { return __uint_as_float((uint32_t)min(266 - ex, 254) << 23); }

__device__ __forceinline__ float row_factor(float to_log2, float up)
{
    // 1 / up by its exponent
    return fmaxf(to_log2 * __uint_as_float((254u << 23) - __float_as_uint(up)), 1e-37f);
}

// the lowest n bits, all for n >= 32, none for n <= 0
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

}  // namespace dspark
