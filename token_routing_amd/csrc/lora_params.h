// Kernel parameter blocks, launch sizes and host launchers of the low-rank
// adapters.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moegg {

// Shrink (in, w -> h) and expand (h, w, base -> out) of T rows; C is the wide
// dimension: columns of `in` or of `out`.
struct LoraParams {
    const uint16_t *in;
    const uint16_t *w;
    const int32_t *m_sizes;
    const int32_t *gather;
    const int32_t *ranks;
    const float *scales;
    const uint16_t *base;
    uint16_t *out;
    float *h;      // [splits][T][R], 8 more values behind
    float *h_out;  // [T][R] the caller's sum of the splits, or null
    int32_t *err;
    int64_t T, ld_in, ld_base, ld_out, split_stride;
    int L, R, C, splits;
    bool scale_shrink;  // the adapter's scale belongs to h (backward), not to out
    bool stream_base;   // base is too large to be worth a place in the caches
    bool copy_unrouted;  // rows of no adapter get base's row, not what out holds
};

struct GradParams {
    LoraParams l;  // m_sizes, gather, ranks, scales, err, T, L
    const uint16_t *x;
    const uint16_t *dy;
    const float *h;
    const float *dh;
    void *dA;
    void *dB;
    float *partials;
    int64_t ld_x, ld_dy;
    int R, K, N, chunk;
    int col_tiles_a, col_tiles_b;  // 128-column tiles of dA and dB (0: not wanted)
    bool fp32_out;
};

// Base and out together past the 256 MB last-level cache: base is then read
// with the nontemporal hint (4096 rows of 28672 columns: 148 -> 138 us the
// call; at 4096 columns, where a projection's output is still cached, the hint
// costs 27.5 -> 32.3 us).
inline bool lora_streams(int64_t T, int C)
{
    return T * C * 4 > ((int64_t)256 << 20);
}

// 16-row blocks of a large shrink tile for ranks up to R: two while the sums
// and the loads in flight fit 128 registers (two workgroups a compute unit).
__host__ __device__ constexpr int shrink_blocks(int R)
{
    return R <= 64 ? 2 : 1;
}

// Tiles are one block of 16 rows, or large where an adapter has 32 rows or more
// on average.
inline bool lora_many_rows(int64_t T, int L)
{
    return T >= 32 * (T < L ? T : L);
}

inline int lora_shrink_rows(int64_t T, int L, int R)
{
    return lora_many_rows(T, L) ? 16 * shrink_blocks(R) : 16;
}

// Shrink splits: how many workgroups share a tile's reduction of C columns.
// One workgroup a compute unit (256) is aimed at, two with ranks above 64, whose
// weights make the reduction longer (rank 128, 4096 rows: 68.7 -> 61.8 us with
// two; 2048 rows at rank 64: 39.7 -> 41.1 us, so one there); a wave's share
// stays at 64 columns or more, and at most 16 partial sums are left to add.
inline int lora_splits(int64_t T, int L, int R, int C)
{
    const int rows = lora_shrink_rows(T, L, R);
    const int64_t tiles = (T + rows - 1) / rows + (T < L ? T : L);
    const int64_t aim = R > 64 ? 512 : 256;
    int64_t n = tiles > 0 ? (aim + tiles - 1) / tiles : 1;
    n = n < C / 512 ? n : C / 512;
    return (int)(n < 1 ? 1 : n > 16 ? 16 : n);
}

// Rank tiles of the gradients, 16 ranks (R <= 16) or 32 each.  64 leave one wave
// a SIMD: at rank 128, 4096 rows, the kernel took 70 us instead of 60.
inline int lora_rank_tiles(int R)
{
    return R <= 32 ? 1 : (R + 31) / 32;
}

// Rows of one chunk of the gradients' reduction, a multiple of 32: such that
// chunks, column tiles and rank tiles make about 384 workgroups (two fit a
// compute unit at a time, and segments that are no whole chunks add some), but
// no fewer than one 32-row step for each of a workgroup's waves.
inline int lora_chunk(int64_t T, int R, int K, int N)
{
    const int64_t tiles = (((int64_t)K + 127) / 128 + ((int64_t)N + 127) / 128) *
                          lora_rank_tiles(R);
    const int64_t c = (T * tiles / 384 + 31) / 32 * 32;
    return (int)(c < 128 ? 128 : c < T ? c : (T + 31) / 32 * 32 + 128);
}

hipError_t lora_shrink_launch(const LoraParams &p, int dtype, bool transposed, hipStream_t stream);
hipError_t lora_expand_launch(const LoraParams &p, int dtype, bool transposed, hipStream_t stream);
hipError_t lora_sum_launch(const float *h, float *out, int64_t n, int splits, hipStream_t stream);
hipError_t lora_grad_launch(const GradParams &p, int dtype, hipStream_t stream);

}  // namespace moegg
