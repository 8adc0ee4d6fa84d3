// Epilogues of the feed-forward block's kernels on the main loop of block_engine.h: a
// lane holds 16 columns of one output row in each 32 x 32 block, and one exchange
// with the lane 32 away makes them two times 8 neighbours (row_cols).  Scales,
// activation, block maxima and codes need no other lane but that one, and a row's 32
// columns leave in whole 32- or 64-byte pieces without shared memory.  Their stores
// are at the memory's rate (8192 x 14336 bf16 of H and twice that of A in 110 us), but
// a compute unit's MFMAs wait for them: with 256 accumulator columns a wave pair
// fills the registers, so that no second tile runs beside.  Tried and slower:
// nontemporal stores (the backward 1.19 -> 1.58 ms: a row's line leaves in pieces),
// groups of workgroups started apart (no gain beyond their delay).
#pragma once

#include <algorithm>
#include <cmath>
#include <utility>

#include "block_engine.h"

#include "block_params.h"
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
// one rounding of the result to bf16.
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

// Row tiles of `rows` rows over E experts, at most.
inline int64_t row_tiles(int64_t rows, int E, int block)
{
    return rows <= E ? rows : (rows - E + 1 + block - 1) / block + E - 1;
}

// Tile shapes: small (32 rows: for a few row tiles of streamed weights), middle (128 x
// 128, two workgroups a compute unit), deep (the same with four stages, one workgroup)
// and large (256 x 256, one).
enum Shape { kSmallTiles, kMidTiles, kDeepTiles, kBigTiles };

// Which of them a launch takes.  Rows per expert are known on the device alone: an
// expert's last row tile counts as half full (one expert's is known).
//   small   where a launch is bound by latency: it has up to `most_small` rounds of
//           small tiles.  8 experts of 64 rows, 2048 into 2048: int8 16.2 us (middle
//           19.5, large 27.8), bf16 23.9 (29.5, 47.6).
//   deep    where the middle tiles leave each compute unit one: nothing else covers
//           a stage's way from memory.  3003 rows of 1008 into 2 x 520, A kept, 18.7 us
//           (middle 21.8); 2048 rows of 2048 into 2 x 768 25.8 (28.1); with 320 tiles for
//           256 units 45.0 (33.5).
//   large   where their rounds over the compute units cost less than the middle
//           tiles', 1.65 times as much a round, two tiles a unit in a middle one whose
//           last round costs what it fills: 60 experts, 2048 into 2048 int8, of 1024
//           rows 318 us (middle 362, small 690), of 128 rows 85 (66, 140).
// 256 x 128 and 128 x 256 tiles with 32-deep stages, two workgroups a unit, lose to
// both (8192 rows of 4096 int8 into 28672 1.19 ms, large 0.98; 65536 of 768 into
// 2048 248 us, large 236).  Swept over 1, 8 and 60 experts of 16 to 1024 rows and 512
// to 8192 columns.
inline Shape tile_shape(int64_t S, int E, int cols, int small_cols, double most_small, int cus)
{
    auto rounds = [&](int64_t bm, int64_t bn, int a_round) {
        const int64_t rows =
            E == 1 ? (S + bm - 1) / bm
                   : std::min(S, std::max(std::min<int64_t>(S, E), S / bm + E / 2));
        return (double)(rows * ((cols + bn - 1) / bn)) / a_round;
    };
    if (rounds(32, small_cols, cus) <= most_small)
        return kSmallTiles;
    const double mid = std::max(0.6, rounds(128, 128, 2 * cus) + 0.2);
    if (1.65 * std::ceil(rounds(256, 256, cus)) < mid)
        return kBigTiles;
    return rounds(128, 128, cus) <= 1.0 ? kDeepTiles : kMidTiles;
}

}  // namespace moegg
