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
// The largest step is 2^121 (b = 248), whose codes are held at +-127, so that no
// value reads back as an infinity: magnitudes from 127.5 * 2^121 on (the largest
// bf16, and the last 2^-8 of fp32's range) come back as 127 * 2^121.
//
// b = 255 marks a block that holds an infinity or NaN: its codes are 0, and
// 0 * 2^128 (infinity's bits) reads back as NaN.
#pragma once

#include "common.h"

namespace moegg {

constexpr uint32_t kAbsBits = 0x7fffffffu, kInfBits = 0x7f800000u;

constexpr uint32_t kLostBlock = 255, kLargestStep = 248;

// The byte of a block whose largest |x| has the bits m: kLargestStep + 1 where
// codes have to be held.
__device__ __forceinline__ uint32_t pack_exp(uint32_t m)
{
    const int b = max((int)((m + 0x10000u) >> 23) - 6, 1);
    return m >= kInfBits ? kLostBlock : (uint32_t)b;
}
__device__ __forceinline__ float pack_step(uint32_t b)
{
    return __uint_as_float(b << 23);
}
// 1 / step, a normal number for every b up to kLargestStep.
__device__ __forceinline__ float pack_inverse(uint32_t b)
{
    return __uint_as_float((254u - b) << 23);
}

// Four codes.  x * inv + 1.5 * 2^23 is rounded to a whole number by the one
// rounding of the fma, and its low byte is the code.
template <bool HOLD>
__device__ __forceinline__ uint32_t pack_code(float x, float inv)
{
    constexpr float kRound = 12582912.0f;
    float r = __builtin_fmaf(x, inv, kRound);
    if constexpr (HOLD)
        r = __builtin_amdgcn_fmed3f(r, kRound - 127.0f, kRound + 127.0f);
    return __float_as_uint(r);
}
template <bool HOLD>
__device__ __forceinline__ uint32_t pack_codes4(float x0, float x1, float x2, float x3, float inv)
{
    const uint32_t lo = __builtin_amdgcn_perm(pack_code<HOLD>(x1, inv), pack_code<HOLD>(x0, inv),
                                              0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(pack_code<HOLD>(x3, inv), pack_code<HOLD>(x2, inv),
                                              0x04000c0cu);
    return lo | hi;
}
// N codes of a block of byte b (pack_exp's), four to a word; b becomes the byte to store.
template <int N>
__device__ __forceinline__ void pack_codes(const float (&f)[N], uint32_t &b, uint32_t (&w)[N / 4])
{
    const float inv = pack_inverse(b);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = pack_codes4<false>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], inv);
    if (b > kLargestStep) {
        const float most = pack_inverse(kLargestStep);
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = b == kLostBlock ? 0u
                                   : pack_codes4<true>(f[4 * i], f[4 * i + 1], f[4 * i + 2],
                                                       f[4 * i + 3], most);
        b = b == kLostBlock ? kLostBlock : kLargestStep;
    }
}

template <int N>
__device__ __forceinline__ uint32_t abs_max_bits(const float (&f)[N])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        m = max(m, __float_as_uint(f[i]) & kAbsBits);
    return m;
}

// 16 columns of a lane and the 16 of the lane 32 away form a block: both get
// its byte, each the codes of its own columns.  All lanes take part.
__device__ __forceinline__ uint32_t pack_cols(const float (&f)[16], uint32_t (&codes)[4])
{
    const uint32_t m = abs_max_bits(f);
    const auto o = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    uint32_t b = pack_exp(max(o[0], o[1]));
    pack_codes(f, b, codes);
    return b;
}

// Codes of columns 8 (l / 32) .. + 7 and 16 + 8 (l / 32) .. + 7 of a block, and of
// columns 16 (l / 32) .. + 15: each is the other's by the same exchange.
__device__ __forceinline__ void exchange_codes(uint32_t (&w)[4])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(w[i], w[2 + i], false, false);
        w[i] = r[0];
        w[2 + i] = r[1];
    }
}

__device__ __forceinline__ void unpack4(uint32_t q, float step, float *f)
{
    f[0] = (float)(int8_t)q * step;
    f[1] = (float)(int8_t)(q >> 8) * step;
    f[2] = (float)(int8_t)(q >> 16) * step;
    f[3] = (float)(int8_t)(q >> 24) * step;
}

// The values of 8 codes.
__device__ __forceinline__ void unpack_cols(uint32_t lo, uint32_t hi, uint32_t b, float (&f)[8])
{
    const float step = pack_step(b);
    unpack4(lo, step, f);
    unpack4(hi, step, f + 4);
}

}  // namespace moegg
