// Epilogues of the feed-forward block's kernels on the main loop of block_engine.h: a
// lane holds 16 columns of one output row in each 32 x 32 block, and one exchange
// with the lane 32 away makes them two times 8 neighbours (row_cols).  Scales,
// activation, block maxima and codes need no other lane but that one, and a row's 32
// columns leave in whole 32- or 64-byte pieces without shared memory.  Their stores
// are at the memory's rate (8192 x 14336 bf16 of H and twice that of A in 110 us), but
// a compute unit's MFMAs wait for them: with 256 accumulator columns a wave pair
// fills the registers, so that no second tile runs beside, and the next tile's first
// waits count the stores (ring_loop).  Tried and slower:
// nontemporal stores (the backward 1.19 -> 1.58 ms: a row's line leaves in pieces),
// groups of workgroups started apart (no gain beyond their delay).
#pragma once

#include <utility>

#include "block_engine.h"

#include "block_params.h"
#include "block_shape.h"
#include "pack.h"

namespace moegg {

// 16 bytes at the alignment of a bf16 (or a byte): global memory takes them so.
typedef unsigned short u16x8_any_t __attribute__((ext_vector_type(8), aligned(2)));

// x of the lanes below 32 with y of those from 32 on: afterwards x holds both
// first halves (x's own, then y's), y both second halves.
__device__ __forceinline__ void swap_halves(uint32_t &x, uint32_t &y)
{
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0];
    y = r[1];
}

// The 16 accumulators of a block as columns of row l % 32: v[8 h + i] is column
// 16 h + 8 (l / 32) + i, so that the two lanes of a row store neighbouring pieces
// with one instruction.  Before, register 4 g + q is column 8 g + 4 (l / 32) + q
// (operands exchanged).
__device__ __forceinline__ int lane_col(int h)
{
    return 16 * h + 8 * ((threadIdx.x & (kWave - 1)) >> 5);
}
__device__ __forceinline__ void row_cols(const f32x16_t &acc, uint32_t (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t x = __float_as_uint(acc[8 * h + q]), y = __float_as_uint(acc[8 * h + 4 + q]);
            swap_halves(x, y);
            v[8 * h + q] = x;
            v[8 * h + 4 + q] = y;
        }
}

// The output: columns as they are, or gated by one of the activations.
constexpr int kPlain = 0, kSilu = 1, kGelu = 2;

// act(g) = g sigmoid(z(g)): z = g for silu, and 2 sqrt(2 / pi) (g + 0.044715 g^3) for
// gelu's tanh form, since (1 + tanh y) / 2 = sigmoid(2 y).  sigmoid(z) = 1 / (1 +
// 2^(-z log2 e)) by v_exp_f32 and v_rcp_f32, good to an ulp each, far below the
// one rounding of the result to bf16.  v_rcp_f32 gives 0 below fp32's normal numbers:
// from z of about -87.3 down, where silu is above -1.1e-36, the activation is 0.
template <bool GELU>
struct GateAct {
    static constexpr float kLog2e = 1.4426950408889634f;
    static constexpr float c0 = 1.5957691216057308f, c1 = 0.07135481627159f;
    static __device__ __forceinline__ float sigmoid(float g)
    {
        const float t = GELU ? g * __builtin_fmaf(-c1 * kLog2e * g, g, -c0 * kLog2e) : g * -kLog2e;
        return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
    }
    static __device__ __forceinline__ float act(float g) { return g * sigmoid(g); }
    // a = act(g) = g s and d = act'(g) = s + g s (1 - s) z'(g).  Gelu's slope is taken
    // at |g| <= 64, beyond which s is 0 or 1 to the last bit: no product overflows
    // (a NaN reaches the result by way of s).
    static __device__ __forceinline__ void slope(float g, float &a, float &d)
    {
        const float s = sigmoid(g);
        a = g * s;
        if constexpr (GELU) {
            const float c = __builtin_amdgcn_fmed3f(g, -64.0f, 64.0f);
            d = __builtin_fmaf(c * s * (1.0f - s), __builtin_fmaf(3.0f * c1 * c, c, c0), s);
        } else {
            d = __builtin_fmaf(a, 1.0f - s, s);
        }
    }
};

// Columns [c, c + 8) of a bf16 row of n elements.  TAIL: n is not a multiple of 8,
// so that a piece may be cut.
template <bool TAIL>
__device__ __forceinline__ void store8(char *row, int c, int n, const float *f)
{
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
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

// The same columns of two planes of width n, as (first, second) neighbours
// (pairs) or as the halves of a row of 2 n.
template <bool TAIL>
__device__ __forceinline__ void store8_planes(char *row, int c, int n, bool halves, const float *f,
                                              const float *s)
{
    if (halves) {
        store8<TAIL>(row, c, n, f);
        store8<TAIL>(row + (int64_t)n * 2, c, n, s);
        return;
    }
    float a[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[2 * i] = f[i];
        a[2 * i + 1] = s[i];
    }
    store8<TAIL>(row, 2 * c, 2 * n, a);
    store8<TAIL>(row, 2 * c + 8, 2 * n, a + 8);
}

template <bool TAIL>
__device__ __forceinline__ u16x8_any_t load8(const char *row, int c, int n)
{
    u16x8_any_t v = {};
    if (c + 8 <= n) {
        v = *reinterpret_cast<const u16x8_any_t *>(row + (int64_t)c * 2);
    } else if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n)
                v[i] = *reinterpret_cast<const uint16_t *>(row + (int64_t)(c + i) * 2);
    }
    return v;
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

}  // namespace moegg
