// Packed activations: blocks of 32 neighbouring values of a row as int8 codes
// with one shared power of two, 8.25 bits a value.
//
// A block's byte is b, its step 2^(b - 127): the smallest for which the block's
// largest magnitude m rounds to at most 127 steps.  m = 1.f * 2^E has 64 to 128
// steps of 2^(E - 6); from 127.5 on (f >= 127/128; the tie rounds to 128) the
// step is one power larger, so E's bits are taken from m's after adding 2^-7 of
// its unit.  A power of two divides without rounding: a code is the one rounding
// (half to even, at most half a step), and code * step has 7 bits, exact in bf16,
// and in fp16 and fp32 inside their ranges.
//
// b = 255 marks a block that holds an infinity or NaN: its codes are 0, and
// 0 * 2^128 (infinity's bits) reads back as NaN.
#pragma once

#include "common.h"

namespace moegg {

constexpr uint32_t kAbsBits = 0x7fffffffu, kInfBits = 0x7f800000u;

// The byte of a block whose largest |x| has the bits m.
__device__ __forceinline__ uint32_t pack_exp(uint32_t m)
{
    const int b = max((int)((m + 0x10000u) >> 23) - 6, 1);
    return m >= kInfBits ? 255u : (uint32_t)b;
}
// 1 / step (0 for a block that is not finite).
__device__ __forceinline__ float pack_inverse(uint32_t b)
{
    return __builtin_bit_cast(float, b == 255u ? 0u : (254u - b) << 23);
}
__device__ __forceinline__ float pack_step(uint32_t b)
{
    return __builtin_bit_cast(float, b << 23);
}

// Four codes.  x * inv + 1.5 * 2^23 is rounded to a whole number by the one
// rounding of the fma, and its low byte is the code.
__device__ __forceinline__ uint32_t pack_codes4(float x0, float x1, float x2, float x3, float inv,
                                                bool finite)
{
    constexpr float kRound = 12582912.0f;
    const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_fmaf(x0, inv, kRound));
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_fmaf(x1, inv, kRound));
    const uint32_t c = __builtin_bit_cast(uint32_t, __builtin_fmaf(x2, inv, kRound));
    const uint32_t d = __builtin_bit_cast(uint32_t, __builtin_fmaf(x3, inv, kRound));
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return finite ? lo | hi : 0u;
}

template <int N>
__device__ __forceinline__ uint32_t abs_max_bits(const float (&f)[N])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        m = max(m, __builtin_bit_cast(uint32_t, f[i]) & kAbsBits);
    return m;
}

// 16 columns of a lane and the 16 of the lane 32 away form a block: both get
// its byte, each the codes of its own columns.  All lanes take part.
__device__ __forceinline__ uint32_t pack_cols(const float (&f)[16], uint4 &codes)
{
    const uint32_t m = abs_max_bits(f);
    const auto o = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    const uint32_t b = pack_exp(max(o[0], o[1]));
    const float inv = pack_inverse(b);
    const bool fin = b != 255u;
    codes.x = pack_codes4(f[0], f[1], f[2], f[3], inv, fin);
    codes.y = pack_codes4(f[4], f[5], f[6], f[7], inv, fin);
    codes.z = pack_codes4(f[8], f[9], f[10], f[11], inv, fin);
    codes.w = pack_codes4(f[12], f[13], f[14], f[15], inv, fin);
    return b;
}

__device__ __forceinline__ void unpack4(uint32_t q, float step, float *f)
{
    f[0] = (float)(int8_t)q * step;
    f[1] = (float)(int8_t)(q >> 8) * step;
    f[2] = (float)(int8_t)(q >> 16) * step;
    f[3] = (float)(int8_t)(q >> 24) * step;
}

__device__ __forceinline__ void unpack_cols(const uint4 &q, uint32_t b, float (&f)[16])
{
    const float step = pack_step(b);
    unpack4(q.x, step, f);
    unpack4(q.y, step, f + 4);
    unpack4(q.z, step, f + 8);
    unpack4(q.w, step, f + 12);
}

}  // namespace moegg
