// Epilogues of the feed-forward block's kernels on the main loop of
// block_engine.h: a lane then holds 16 columns of
// one output row in each 32 x 32 block, and one exchange with the lane 32 away
// makes them 16 neighbours (row_cols).  Scales, activation, block maxima and codes
// need no other lane but that one, and a row's 32 columns leave in whole 32- or
// 64-byte pieces without shared memory.
#pragma once

#include <algorithm>
#include <utility>

#include "block_engine.h"

#include "block_params.h"
#include "pack.h"

namespace moegg {

typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at the alignment of a bf16 (or a byte): global memory takes them so.
typedef unsigned short u16x8_any_t __attribute__((ext_vector_type(8), aligned(2)));
typedef unsigned u32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

// x of the lanes below 32 with y of those from 32 on: afterwards x holds both
// first halves (x's own, then y's), y both second halves.
__device__ __forceinline__ void swap_halves(uint32_t &x, uint32_t &y)
{
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}

// The 16 accumulators of a block as neighbouring columns: lane l holds columns
// 16 (l / 32) .. + 15 of row l % 32.  Before, register 4 g + q is column
// 8 g + 4 (l / 32) + q (operands exchanged).
__device__ __forceinline__ void row_cols(const f32x16_t &acc, uint32_t (&v)[16])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t x0 = __float_as_uint(acc[q]), x1 = __float_as_uint(acc[4 + q]);
        uint32_t x2 = __float_as_uint(acc[8 + q]), x3 = __float_as_uint(acc[12 + q]);
        swap_halves(x0, x2);
        swap_halves(x1, x3);
        v[q] = x0;
        v[4 + q] = x2;
        v[8 + q] = x1;
        v[12 + q] = x3;
    }
}

// The activation's argument z(g) = g (c0 + c1 g^2) of the sigmoid: silu is g
// sigmoid(g), and gelu's tanh form g sigmoid(z), for which (1 + tanh y) / 2 =
// sigmoid(2 y) with y = sqrt(2 / pi) (g + 0.044715 g^3).  v_exp_f32 and
// v_rcp_f32 are good to an ulp, far below the one rounding of the result to bf16.
struct GateAct {
    float c0, c1;
    __device__ __forceinline__ explicit GateAct(bool gelu)
        : c0(gelu ? 1.5957691216057308f : 1.0f), c1(gelu ? 0.07135481627159f : 0.0f)
    {
    }
    __device__ __forceinline__ float sigmoid(float g) const
    {
        const float z = g * __builtin_fmaf(c1 * g, g, c0);
        return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    }
    __device__ __forceinline__ float operator()(float g) const { return g * sigmoid(g); }
    // act(g) = g s and act'(g) = s + g s (1 - s) z'(g).  Beyond |g| = 64 s is 0 or
    // 1 to the last bit, so that the slope is taken there, where no product
    // overflows (a NaN goes through the clamp's result by way of s).
    __device__ __forceinline__ void slope(float g, float &a, float &d) const
    {
        const float s = sigmoid(g);
        const float c = __builtin_amdgcn_fmed3f(g, -64.0f, 64.0f);
        const float dz = __builtin_fmaf(3.0f * c1 * c, c, c0);
        a = g * s;
        d = __builtin_fmaf(c * s * (1.0f - s), dz, s);
    }
};

// Columns [col, col + 16) of a bf16 row of n elements.  TAIL: n is not a multiple
// of 8, so that a piece may be cut.
template <bool TAIL>
__device__ __forceinline__ void store_cols(char *row, int col, int n, const float (&f)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = col + 8 * h;
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2(f[8 * h + 2 * i], f[8 * h + 2 * i + 1]);
        const u16x8_any_t v = __builtin_bit_cast(u16x8_any_t, w);
        if (c + 8 <= n) {
            *reinterpret_cast<u16x8_any_t *>(row + (int64_t)c * 2) = v;
        } else if constexpr (TAIL) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < n)
                    *reinterpret_cast<uint16_t *>(row + (int64_t)(c + i) * 2) = v[i];
        }
    }
}

// The same columns of two planes of width n, as (first, second) neighbours
// (pairs) or as the halves of a row of 2 n.
template <bool TAIL>
__device__ __forceinline__ void store_planes(char *row, int col, int n, bool halves,
                                             const float (&f)[16], const float (&s)[16])
{
    if (halves) {
        store_cols<TAIL>(row, col, n, f);
        store_cols<TAIL>(row + (int64_t)n * 2, col, n, s);
        return;
    }
    float a[16], b[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[2 * i] = f[i];
        a[2 * i + 1] = s[i];
        b[2 * i] = f[8 + i];
        b[2 * i + 1] = s[8 + i];
    }
    store_cols<TAIL>(row, 2 * col, 2 * n, a);
    store_cols<TAIL>(row, 2 * col + 16, 2 * n, b);
}

template <bool TAIL>
__device__ __forceinline__ void load_cols(const char *row, int col, int n, float (&f)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = col + 8 * h;
        u16x8_any_t v = {};
        if (c + 8 <= n) {
            v = *reinterpret_cast<const u16x8_any_t *>(row + (int64_t)c * 2);
        } else if constexpr (TAIL) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < n)
                    v[i] = *reinterpret_cast<const uint16_t *>(row + (int64_t)(c + i) * 2);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[8 * h + i] = __uint_as_float((uint32_t)v[i] << 16);
    }
}

template <bool TAIL>
__device__ __forceinline__ void load_planes(const char *row, int col, int n, bool halves,
                                            float (&f)[16], float (&s)[16])
{
    if (halves) {
        load_cols<TAIL>(row, col, n, f);
        load_cols<TAIL>(row + (int64_t)n * 2, col, n, s);
        return;
    }
    float a[16], b[16];
    load_cols<TAIL>(row, 2 * col, 2 * n, a);
    load_cols<TAIL>(row, 2 * col + 16, 2 * n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = a[2 * i];
        s[i] = a[2 * i + 1];
        f[8 + i] = b[2 * i];
        s[8 + i] = b[2 * i + 1];
    }
}

// f(i) for the constants i = 0 .. N - 1: an epilogue's block indices have to be
// constants whatever its size (accumulators indexed by a variable live in memory).
template <class F, int... I>
__device__ __forceinline__ void for_constants(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void for_constants(F f)
{
    for_constants(std::make_integer_sequence<int, N>{}, f);
}

// Workgroups of a kernel that a compute unit holds.
template <class Kern>
int resident_workgroups(Kern kernel, int threads)
{
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != hipSuccess || n < 1)
        n = 1;
    return n;
}

// Row tiles of `rows` rows over E experts, at most.
inline int64_t row_tiles(int64_t rows, int E, int block)
{
    return rows <= E ? rows : (rows - E + 1 + block - 1) / block + E - 1;
}

// Average rows per expert below which the small tiles are used, as for the
// bf16 products.
constexpr int64_t kBlockSmallRows = 96;

}  // namespace moegg
