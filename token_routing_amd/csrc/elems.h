// Typed element access for the kernels that take bf16, fp16 or fp32 rows.
//
// A lane moves 16 bytes (8 elements of 16 bits, 4 of 32): global memory takes
// 16-byte accesses at element alignment on gfx950, so odd row lengths use the
// same accesses and only the row's last, partial piece goes by elements.
#pragma once

#include "common.h"

namespace moegg {

// Element types (mirrors MOEGG_BF16, MOEGG_FP16, MOEGG_FP32 in moegg.h).
constexpr int kBf16 = 0;
constexpr int kFp16 = 1;
constexpr int kFp32 = 2;

template <int DT> struct Elem;

template <> struct Elem<kBf16> {
    typedef uint16_t store_t;
    static constexpr int kPer16 = 8;
    static __device__ __forceinline__ float widen(store_t v)
    {
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    }
    static __device__ __forceinline__ store_t narrow(float f) { return to_bf16(f); }
};

template <> struct Elem<kFp16> {
    typedef uint16_t store_t;
    static constexpr int kPer16 = 8;
    static __device__ __forceinline__ float widen(store_t v)
    {
        return (float)__builtin_bit_cast(_Float16, v);
    }
    // The fp32 value is kept apart from the product or sum that made it: the
    // compiler would fuse the two into a mixed-precision fma that rounds once,
    // where the other types round to fp32 first.
    static __device__ __forceinline__ store_t narrow(float f)
    {
        asm("" : "+v"(f));
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    }
};

template <> struct Elem<kFp32> {
    typedef float store_t;
    static constexpr int kPer16 = 4;
    static __device__ __forceinline__ float widen(store_t v) { return v; }
    static __device__ __forceinline__ store_t narrow(float f) { return f; }
};

// 16 bytes of elements, with the alignment of one element.
template <int DT> struct Pack16 {
    typedef typename Elem<DT>::store_t vec_t
        __attribute__((ext_vector_type(Elem<DT>::kPer16), aligned(sizeof(typename Elem<DT>::store_t))));
};

template <int DT, int N>
__device__ __forceinline__ void widen_all(float (&f)[N], const typename Pack16<DT>::vec_t &v)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = Elem<DT>::widen(v[i]);
}

// row[col .. col + 16 bytes) of a row of n elements; elements at or past n read as 0.
template <int DT>
__device__ __forceinline__ typename Pack16<DT>::vec_t
load16(const typename Elem<DT>::store_t *row, int col, int n)
{
    typedef typename Pack16<DT>::vec_t vec_t;
    constexpr int P = Elem<DT>::kPer16;
    if (col + P <= n)
        return *reinterpret_cast<const vec_t *>(row + col);
    vec_t v = {};
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (col + i < n)
            v[i] = row[col + i];
    return v;
}

template <int DT, bool STREAM = true>
__device__ __forceinline__ void store16(typename Elem<DT>::store_t *row, int col, int n,
                                        const float *f)
{
    typedef typename Pack16<DT>::vec_t vec_t;
    constexpr int P = Elem<DT>::kPer16;
    vec_t v;
#pragma unroll
    for (int i = 0; i < P; ++i)
        v[i] = Elem<DT>::narrow(f[i]);
    if (col + P <= n) {
        if constexpr (STREAM)
            __builtin_nontemporal_store(v, reinterpret_cast<vec_t *>(row + col));
        else
            *reinterpret_cast<vec_t *>(row + col) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (col + i < n)
            row[col + i] = v[i];
}

}  // namespace moegg
