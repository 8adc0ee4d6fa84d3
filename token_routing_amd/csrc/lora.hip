// Low-rank adapters of many requests beside a shared projection, gfx950.
//
//   forward   h[p] = x[src(p)] A_a^T                      (shrink)
//             y[src(p)] = base[src(p)] + s_a h[p] B_a^T   (expand)
//   backward  dh[p] = s_a dy[src(p)] B_a                  (shrink, B transposed)
//             dx[src(p)] = base[src(p)] + dh[p] A_a       (expand, A transposed)
//             dA_a = sum_p dh[p]^T x[src(p)], dB_a = s_a sum_p dy[src(p)]^T h[p]  (grad)
//
// for sorted position p of adapter a.  With ranks of 4 to 256 against rows of
// thousands of columns every one of these is bound by moving x, y and dy, so
// the matrix instructions (16 x 16 x 32, fp32 accumulators) read their
// fragments straight from global memory, with no LDS staging: a lane's 8
// reduction elements are 16 contiguous bytes.
//
// Operands whose reduction runs along a strided index (B in dh, A in dx, x and
// dy in the gradients) are loaded as 8 rows of up to 8 contiguous elements a
// lane and transposed in registers, two 16-bit halves per byte permute.  The
// reduction order inside an instruction is free as long as both operands
// agree, and so is the assignment of output rows to lanes; it is chosen so
// that a lane's outputs are 16 contiguous bytes and four lanes' 64.
//
// h and dh stay in fp32 between the kernels.  Where one enters a matrix
// instruction it goes as the sum of two 16-bit values (high part and rounded
// rest), which keeps 16 bits of mantissa in bf16 and 22 in fp16, at twice the
// matrix instructions, of which there are few.  With ranks up to 16 both parts
// share one instruction: its 32 reduction elements hold 16 high and 16 low
// ones.  fp16 parts are scaled by a power of two first, so that values past
// the type's range survive.
//
// Rows go by tiles inside one adapter's segment; each wave finds its tile by
// a scan of m_sizes in registers (64 segments a step), so no launch depends
// on the host knowing the sizes.
#include "elems.h"

#include "lora_params.h"

namespace moegg {

namespace {

constexpr int kErrRank = 16;  // MOEGG_DERR_RANK

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- tiles

struct Tile {
    int a;      // adapter
    int p0;     // first sorted position
    int rows;   // rows of the tile
    int m;      // rows of the adapter
    int index;  // tile number inside the adapter
    int slot;   // partial sums' first place (segments of several tiles only)
};

// Sums saturate at S, so that bad sizes cannot wrap around.
__device__ __forceinline__ uint32_t scan_rows(uint32_t v, uint32_t S)
{
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = __shfl_up(v, d, kWave);
        if (lane >= d)
            v = min(v + o, S);
    }
    return v;
}
__device__ __forceinline__ int scan_sum(int v)
{
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(v, d, kWave);
        if (lane >= d)
            v += o;
    }
    return v;
}

// The tile `want` of all segments' tiles of `per` rows (empty segments have
// `empty` tiles); false past the last one.  By adapter with by_adapter: the
// segment of adapter `want`.  All lanes of the wave call it.
__device__ __forceinline__ bool find_tile(const int32_t *m_sizes, int L, uint32_t S, int want,
                                          int per, int empty, bool by_adapter, Tile &t)
{
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t row0 = 0;
    int tile0 = 0, slot0 = 0;
    for (int c = 0; c < L; c += kWave) {
        const int a = c + lane;
        const int raw = a < L ? m_sizes[a] : 0;
        const uint32_t v = min((uint32_t)max(raw, 0), S);
        const uint32_t end = min(scan_rows(v, S) + row0, S);
        uint32_t start = __shfl_up(end, 1, kWave);
        if (lane == 0)
            start = row0;
        const int m = (int)(end - start);
        const int n = m > 0 ? (m - 1) / per + 1 : (a < L ? empty : 0);
        const int tiles = scan_sum(n);
        const int slots = scan_sum(n > 1 ? n : 0);
        const uint64_t hit =
            __ballot(by_adapter ? a == want : a < L && tile0 + tiles > want);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            t.a = c + l;
            t.m = __shfl(m, l, kWave);
            t.index = by_adapter ? 0 : want - (tile0 + __shfl(tiles - n, l, kWave));
            t.p0 = (int)__shfl(start, l, kWave) + t.index * per;
            t.rows = min(per, t.m - t.index * per);
            t.slot = slot0 + __shfl(slots, l, kWave) - (t.m > per ? (t.m - 1) / per + 1 : 0);
            return true;
        }
        row0 = __shfl(end, kWave - 1, kWave);
        tile0 += __shfl(tiles, kWave - 1, kWave);
        slot0 += __shfl(slots, kWave - 1, kWave);
    }
    return false;
}

// One wave of a launch reports sizes and ranks out of range.
__device__ __forceinline__ void check_sizes(const int32_t *m_sizes, const int32_t *ranks, int L,
                                            int64_t S, int R, int32_t *err)
{
    if (!err || blockIdx.x != 0 || threadIdx.x >= kWave)
        return;
    int64_t sum = 0;
    bool bad = false, bad_rank = false;
    for (int a = threadIdx.x; a < L; a += kWave) {
        bad |= m_sizes[a] < 0;
        sum += max(m_sizes[a], 0);
        if (ranks)
            bad_rank |= ranks[a] < 0 || ranks[a] > R;
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1)
        sum += __shfl_xor((long long)sum, d, kWave);
    if (bad || sum > S)
        raise_error(err, kErrMSizes);
    if (bad_rank)
        raise_error(err, kErrRank);
}

__device__ __forceinline__ int rank_of(const int32_t *ranks, int a, int R)
{
    return ranks ? min(max(ranks[a], 0), R) : R;
}

// Row of x, y or dy at sorted position p (-1: a bad gather entry).
__device__ __forceinline__ int64_t source_row(const LoraParams &a, int p)
{
    if (!a.gather)
        return p;
    const int r = a.gather[p];
    if (r < 0 || r >= a.T) {
        raise_error(a.err, kErrGather);
        return -1;
    }
    return r;
}

// ---------------------------------------------------------------- fragments

template <int DT>
__device__ __forceinline__ f32x4_t mfma(const u32x4_t &a, const u32x4_t &b, const f32x4_t &c)
{
    if constexpr (DT == kBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Elements [col, col + 8) of a 16-bit row of n elements (0 past n; row may be null).
__device__ __forceinline__ u32x4_t load8(const uint16_t *row, int col, int n)
{
    typedef Pack16<kBf16>::vec_t vec_t;
    if (!row)
        return u32x4_t{};
    const vec_t v = load16<kBf16>(row, col, n);
    return __builtin_bit_cast(u32x4_t, v);
}

// Elements [col, col + W) as packed pairs; those at or past n read as 0.
template <int W>
__device__ __forceinline__ void load_pairs(uint32_t (&d)[W < 2 ? 1 : W / 2], const uint16_t *row,
                                           int col, int n, bool on)
{
    typedef uint16_t vec_t __attribute__((ext_vector_type(W), aligned(2)));
    constexpr int D = W < 2 ? 1 : W / 2;
#pragma unroll
    for (int i = 0; i < D; ++i)
        d[i] = 0;
    if (!on || col >= n)
        return;
    if constexpr (W == 1) {
        d[0] = row[col];
    } else {
        if (col + W <= n) {
            const vec_t v = *reinterpret_cast<const vec_t *>(row + col);
#pragma unroll
            for (int i = 0; i < D; ++i)
                d[i] = (uint32_t)v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
            return;
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (col + i < n)
                d[i / 2] |= (uint32_t)row[col + i] << (16 * (i & 1));
    }
}

// Fragment j of 8 rows of W elements: element j of each row, row order.
template <int W>
__device__ __forceinline__ u32x4_t column(const uint32_t (&rows)[8][W < 2 ? 1 : W / 2], int j)
{
    u32x4_t f;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        f[d] = __builtin_amdgcn_perm(rows[2 * d + 1][j / 2], rows[2 * d][j / 2],
                                     (j & 1) ? 0x07060302u : 0x05040100u);
    return f;
}

// A power of two that brings values of magnitude up to `top` into fp16's range.
__device__ __forceinline__ float fit_scale(float top)
{
    const int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23);  // top >= 0
    const int shift = (e == 0 || e == 255) ? 127 : min(max(127 + 14 + 127 - e, 1), 253);
    return __builtin_bit_cast(float, (uint32_t)shift << 23);
}
__device__ __forceinline__ float inverse_scale(float s)
{
    return __builtin_bit_cast(float, (uint32_t)(254 - (__builtin_bit_cast(uint32_t, s) >> 23)) << 23);
}

// v as high + low 16-bit parts.  A value that is not finite has no rest.
template <int DT>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4_t &hi, u32x4_t &lo)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        float h[2], r[2];
        if constexpr (DT == kBf16) {
            hi[d] = pack_bf16x2(v[2 * d], v[2 * d + 1]);
            h[0] = __builtin_bit_cast(float, hi[d] << 16);
            h[1] = __builtin_bit_cast(float, hi[d] & 0xffff0000u);
        } else {
            const uint32_t a = Elem<kFp16>::narrow(v[2 * d]), b = Elem<kFp16>::narrow(v[2 * d + 1]);
            hi[d] = a | b << 16;
            h[0] = Elem<kFp16>::widen((uint16_t)a);
            h[1] = Elem<kFp16>::widen((uint16_t)b);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = fabsf(h[i]) < __builtin_huge_valf() ? v[2 * d + i] - h[i] : 0.0f;
        if constexpr (DT == kBf16)
            lo[d] = pack_bf16x2(r[0], r[1]);
        else
            lo[d] = (uint32_t)Elem<kFp16>::narrow(r[0]) | (uint32_t)Elem<kFp16>::narrow(r[1]) << 16;
    }
}

// h[p][col .. col + 8), the splits' partial sums added in order (0 past n).
__device__ __forceinline__ void load_h(float (&v)[8], const float *h, int64_t p, int R, int col,
                                       int n, int splits, int64_t split_stride, bool on)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = 0.0f;
    if (!on || col >= n)
        return;
    const float *q = h + p * R + col;
    for (int s = 0; s < splits; ++s, q += split_stride) {
        if (col + 8 <= n) {
            const f32x4u_t a = *reinterpret_cast<const f32x4u_t *>(q);
            const f32x4u_t b = *reinterpret_cast<const f32x4u_t *>(q + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += a[i];
                v[4 + i] += b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < n)
                    v[i] += q[i];
        }
    }
}

// ---------------------------------------------------------------- shrink

// h[p, r] = factor * sum_c in[src(p), c] * w(r, c) for a tile of 16 rows:
// w(r, c) = W[r][c] (W [R, C], forward) or W[c][r] (W [C, R], TR).  A
// workgroup of 8 waves takes 1 / splits of the reduction, each wave an equal
// run of it, and adds the waves' sums through LDS in wave order.  Unsplit, the
// sums go to H, else to the split's own copy.  RF: 16-row blocks of ranks.
constexpr int kShrinkWaves = 8;

template <int DT, bool TR, int RF>
__global__ __launch_bounds__(kShrinkWaves *kWave) void shrink_kernel(LoraParams a)
{
    constexpr int W = RF;  // ranks a lane holds with TR: r = m * RF + j
    __shared__ f32x4_t s_acc[kShrinkWaves / 2][RF][kWave];
    check_sizes(a.m_sizes, a.ranks, a.L, a.T, a.R, a.err);
    const int split = blockIdx.x % a.splits;
    Tile tile;
    if (!find_tile(a.m_sizes, a.L, (uint32_t)a.T, blockIdx.x / a.splits, kShrinkRows, 0, false,
                   tile))
        return;
    const int rank = rank_of(a.ranks, tile.a, a.R);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int m = lane & 15, g = lane >> 4;

    const uint16_t *row = nullptr;
    if (m < tile.rows) {
        const int64_t r = source_row(a, tile.p0 + m);
        row = r < 0 ? nullptr : a.in + r * a.ld_in;
    }
    const uint16_t *const w = a.w + (int64_t)tile.a * a.R * a.C;

    f32x4_t acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f)
        acc[f] = f32x4_t{};
    const int steps = (a.C + 31) / 32;
    const int parts = a.splits * kShrinkWaves;
    const int part = split * kShrinkWaves + wave;
    const int s0 = (int)((int64_t)steps * part / parts);
    const int s1 = (int)((int64_t)steps * (part + 1) / parts);
    if (rank > 0) {
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const int c = s * 32 + g * 8;
            const u32x4_t x = load8(row, c, a.C);
            if constexpr (!TR) {
#pragma unroll
                for (int f = 0; f < RF; ++f) {
                    const int r = f * 16 + m;
                    const u32x4_t v = load8(r < rank ? w + (int64_t)r * a.C : nullptr, c, a.C);
                    acc[f] = mfma<DT>(v, x, acc[f]);
                }
            } else {
                uint32_t v[8][W < 2 ? 1 : W / 2];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    load_pairs<W>(v[e], w + (int64_t)(c + e) * a.R, m * W, rank, c + e < a.C);
#pragma unroll
                for (int f = 0; f < RF; ++f)
                    acc[f] = mfma<DT>(column<W>(v, f), x, acc[f]);
            }
        }
    }
#pragma unroll
    for (int half = kShrinkWaves / 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int f = 0; f < RF; ++f)
                s_acc[wave - half][f][lane] = acc[f];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int f = 0; f < RF; ++f)
                acc[f] += s_acc[wave][f][lane];
        __syncthreads();
    }
    if (wave != 0 || m >= tile.rows)
        return;
    const float factor = a.scale_shrink && a.scales ? a.scales[tile.a] : 1.0f;
    float *const h = a.h + split * a.split_stride + (int64_t)(tile.p0 + m) * a.R;
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = TR ? (4 * g + i) * RF + f : f * 16 + 4 * g + i;
            if (r < a.R)
                h[r] = factor * acc[f][i];
        }
}

// ---------------------------------------------------------------- expand

// out[src(p), c] = base[src(p), c] + factor * sum_r h[p, r] * w(r, c), w(r, c)
// = W[c][r] (W [C, R], forward) or W[r][c] (W [R, C], TR).  A wave takes RT *
// 16 rows of one adapter and F * 16 columns; its weights' fragments are loaded
// once for all of its rows.  SMALL: ranks up to 16, both parts of h in one
// instruction.
template <int DT, bool TR, bool SMALL>
__global__ __launch_bounds__(256) void expand_kernel(LoraParams a, int col_tiles)
{
    constexpr int F = TR ? 8 : 4;
    constexpr int RT = TR ? kExpandRowsT / 16 : kExpandRows / 16;
    constexpr int kRows = RT * 16;
    constexpr int kCols = F * 16;
    constexpr int kStep = SMALL ? 16 : 32;
    check_sizes(a.m_sizes, a.ranks, a.L, a.T, a.R, a.err);
    Tile tile;
    if (!find_tile(a.m_sizes, a.L, (uint32_t)a.T, blockIdx.x / col_tiles, kRows, 0, false, tile))
        return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int m = lane & 15, g = lane >> 4;
    const int col_tile = blockIdx.x % col_tiles;
    const int c0 = (col_tile * 4 + wave) * kCols;
    const int rank = rank_of(a.ranks, tile.a, a.R);
    const int rg = SMALL ? (g & 1) * 8 : g * 8;  // this lane's ranks of a step

    // The summed h for the caller, by the first column tile.
    if (a.h_out && col_tile == 0)
        for (int i = threadIdx.x; i < tile.rows * a.R; i += 256) {
            const float *q = a.h + (int64_t)tile.p0 * a.R + i;
            float v = 0.0f;
            for (int s = 0; s < a.splits; ++s, q += a.split_stride)
                v += *q;
            a.h_out[(int64_t)tile.p0 * a.R + i] = v;
        }
    if (c0 >= a.C || (rank == 0 && a.base == a.out))
        return;
    const uint16_t *const w = a.w + (int64_t)tile.a * a.R * a.C;

    f32x4_t acc[RT][F];
    float fit[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        fit[t] = 1.0f;
#pragma unroll
        for (int f = 0; f < F; ++f)
            acc[t][f] = f32x4_t{};
    }
    if constexpr (DT == kFp16) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float top = 0.0f, v[8];
            for (int r = 0; r < rank; r += kStep) {
                load_h(v, a.h, tile.p0 + t * 16 + m, a.R, r + rg, rank, a.splits, a.split_stride,
                       t * 16 + m < tile.rows);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = fmaxf(top, fabsf(v[i]));
            }
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            fit[t] = fit_scale(top);
        }
    }
    for (int r0 = 0; r0 < rank; r0 += kStep) {
        u32x4_t wf[F];
        if constexpr (TR) {
            uint32_t v[8][4];
            const int c = c0 + ((m & 3) * 4 + (m >> 2)) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                load_pairs<8>(v[e], w + (int64_t)(r0 + rg + e) * a.C, c, a.C, r0 + rg + e < rank);
#pragma unroll
            for (int f = 0; f < F; ++f)
                wf[f] = column<8>(v, f);
        } else {
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int c = c0 + (f >> 1) * 32 + (m >> 2) * 8 + (f & 1) * 4 + (m & 3);
                wf[f] = load8(c < a.C ? w + (int64_t)c * a.R : nullptr, r0 + rg, rank);
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (t * 16 >= tile.rows)
                break;
            float v[8];
            u32x4_t hi, lo;
            load_h(v, a.h, tile.p0 + t * 16 + m, a.R, r0 + rg, rank, a.splits, a.split_stride,
                   t * 16 + m < tile.rows);
            if constexpr (DT == kFp16)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] *= fit[t];
            split8<DT>(v, hi, lo);
            if constexpr (SMALL) {
                const u32x4_t both = g < 2 ? hi : lo;
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc[t][f] = mfma<DT>(wf[f], both, acc[t][f]);
            } else {
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    acc[t][f] = mfma<DT>(wf[f], hi, acc[t][f]);
                    acc[t][f] = mfma<DT>(wf[f], lo, acc[t][f]);
                }
            }
        }
    }
    const float factor = !a.scale_shrink && a.scales ? a.scales[tile.a] : 1.0f;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if (t * 16 + m >= tile.rows)
            continue;
        const int64_t row = source_row(a, tile.p0 + t * 16 + m);
        if (row < 0)
            continue;
        const uint16_t *const base = a.base + row * a.ld_base;
        uint16_t *const out = a.out + row * a.ld_out;
        const float k = DT == kFp16 ? factor * inverse_scale(fit[t]) : factor;
        constexpr int kPieces = TR ? 4 : 2;
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int c = TR ? c0 + (q * 4 + g) * 8 : c0 + q * 32 + g * 8;
            float y[8];
            if (c >= a.C)
                continue;
            widen_all<DT>(y, load16<DT>(base, c, a.C));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = TR ? acc[t][TR ? i : 0][q] : acc[t][TR ? 0 : 2 * q + (i >> 2)][i & 3];
                y[i] += k * d;
            }
            store16<DT>(out, c, a.C, y);
        }
    }
}

// ---------------------------------------------------------------- grad

// G[c, r] = factor * sum_p big[src(p), c] * small[p, r] over a chunk of one
// adapter's rows: dA (big = x, small = dh; stored [r][c]) in the first
// col_tiles_a column tiles, dB (big = dy, small = h; stored [c][r]) in the
// rest.  A workgroup of 4 waves takes 128 columns and RG * 16 ranks; the waves
// take turns at 32-row steps and add their sums through LDS.  A segment of
// one chunk is finished here, the others leave fp32 partials.
template <int DT, int RG>
__global__ __launch_bounds__(256) void grad_kernel(GradParams a)
{
    __shared__ f32x4_t s_acc[2][8 * RG][kWave];
    const int rank_tiles = (a.R + RG * 16 - 1) / (RG * 16);
    const int tiles = a.col_tiles_a + a.col_tiles_b;
    int b = blockIdx.x;
    const int rt = b % rank_tiles;
    b /= rank_tiles;
    int ct = b % tiles;
    Tile tile;
    if (!find_tile(a.l.m_sizes, a.l.L, (uint32_t)a.l.T, b / tiles, a.chunk, 1, false, tile))
        return;
    const bool is_a = ct < a.col_tiles_a;
    ct -= is_a ? 0 : a.col_tiles_a;
    const int C = is_a ? a.K : a.N;
    const uint16_t *const big = is_a ? a.x : a.dy;
    const int64_t ld = is_a ? a.ld_x : a.ld_dy;
    const float *const small = is_a ? a.dh : a.h;
    const int splits = is_a ? a.splits : 1;
    const int rank = rank_of(a.l.ranks, tile.a, a.R);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int m = lane & 15, g = lane >> 4;
    const int c_load = ct * 128 + ((m & 3) * 4 + (m >> 2)) * 8;
    const int r0 = rt * RG * 16 + m;

    auto load_small = [&](float (&v)[8], int p, int end, int r) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = 0.0f;
            if (r < rank && p + e < end) {
                const float *q = small + (int64_t)(p + e) * a.R + r;
                for (int s = 0; s < splits; ++s, q += a.split_stride)
                    v[e] += *q;
            }
        }
    };

    f32x4_t acc[8][RG];
    float fit[RG];
#pragma unroll
    for (int q = 0; q < RG; ++q) {
        fit[q] = 1.0f;
#pragma unroll
        for (int f = 0; f < 8; ++f)
            acc[f][q] = f32x4_t{};
    }
    const int end = tile.p0 + max(tile.rows, 0);
    if constexpr (DT == kFp16) {
        float top[RG] = {};
        for (int p = tile.p0 + wave * 32; p < end; p += 128)
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                float v[8];
                load_small(v, p + g * 8, end, r0 + q * 16);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top[q] = fmaxf(top[q], fabsf(v[e]));
            }
#pragma unroll
        for (int q = 0; q < RG; ++q) {
            top[q] = fmaxf(top[q], __shfl_xor(top[q], 16, kWave));
            top[q] = fmaxf(top[q], __shfl_xor(top[q], 32, kWave));
            fit[q] = fit_scale(top[q]);
        }
    }
    for (int p = tile.p0 + wave * 32; p < end; p += 128) {
        uint32_t v[8][4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = p + g * 8 + e;
            const int64_t row = at < end ? source_row(a.l, at) : -1;
            load_pairs<8>(v[e], big + (row < 0 ? 0 : row) * ld, c_load, C, row >= 0);
        }
        u32x4_t hi[RG], lo[RG];
#pragma unroll
        for (int q = 0; q < RG; ++q) {
            float s[8];
            load_small(s, p + g * 8, end, r0 + q * 16);
            if constexpr (DT == kFp16)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[e] *= fit[q];
            split8<DT>(s, hi[q], lo[q]);
        }
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            const u32x4_t bf = column<8>(v, f);
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                acc[f][q] = mfma<DT>(bf, hi[q], acc[f][q]);
                acc[f][q] = mfma<DT>(bf, lo[q], acc[f][q]);
            }
        }
    }
    if constexpr (DT == kFp16) {
#pragma unroll
        for (int q = 0; q < RG; ++q)
#pragma unroll
            for (int f = 0; f < 8; ++f)
                acc[f][q] *= inverse_scale(fit[q]);
    }
#pragma unroll
    for (int half = 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int f = 0; f < 8; ++f)
#pragma unroll
                for (int q = 0; q < RG; ++q)
                    s_acc[wave - half][f * RG + q][lane] = acc[f][q];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int f = 0; f < 8; ++f)
#pragma unroll
                for (int q = 0; q < RG; ++q)
                    acc[f][q] += s_acc[wave][f * RG + q][lane];
        __syncthreads();
    }
    if (wave != 0)
        return;
    const float factor = !is_a && a.l.scales ? a.l.scales[tile.a] : 1.0f;
    const bool whole = tile.m <= a.chunk;
    const int64_t size_a = (int64_t)a.R * a.K;
    float *const part = a.partials + (int64_t)(tile.slot + tile.index) * ((a.K + (int64_t)a.N) * a.R) +
                        (is_a ? 0 : size_a);
    char *const out = static_cast<char *>(is_a ? a.dA : a.dB);
    const int64_t out0 = (int64_t)tile.a * a.R * C;
#pragma unroll
    for (int q = 0; q < RG; ++q) {
        const int r = r0 + q * 16;
        if (r >= a.R)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = ct * 128 + (i * 4 + g) * 8;
#pragma unroll
            for (int f = 0; f < 8; ++f) {
                if (c + f >= C)
                    continue;
                const int64_t at = is_a ? (int64_t)r * C + c + f : (int64_t)(c + f) * a.R + r;
                const float v = factor * acc[f][q][i];
                if (!whole)
                    part[at] = v;
                else if (a.fp32_out)
                    reinterpret_cast<float *>(out)[out0 + at] = v;
                else
                    reinterpret_cast<uint16_t *>(out)[out0 + at] = Elem<DT>::narrow(v);
            }
        }
    }
}

// Adds the partials of adapters with several chunks, in chunk order.
template <int DT>
__global__ __launch_bounds__(256) void grad_join_kernel(GradParams a, int blocks)
{
    Tile tile;
    if (!find_tile(a.l.m_sizes, a.l.L, (uint32_t)a.l.T, blockIdx.x / blocks, a.chunk, 1, true,
                   tile) ||
        tile.m <= a.chunk)
        return;
    const int chunks = (tile.m - 1) / a.chunk + 1;
    const int64_t size_a = (int64_t)a.R * a.K, size = size_a + (int64_t)a.R * a.N;
    const float *const part = a.partials + (int64_t)tile.slot * size;
    for (int64_t i = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x; i < size;
         i += (int64_t)blocks * 256) {
        const bool is_a = i < size_a;
        void *const out = is_a ? a.dA : a.dB;
        float v = 0.0f;
        for (int c = 0; c < chunks; ++c)
            v += part[c * size + i];
        const int64_t at = is_a ? (int64_t)tile.a * size_a + i
                                : (int64_t)tile.a * a.R * a.N + (i - size_a);
        if (a.fp32_out)
            static_cast<float *>(out)[at] = v;
        else
            static_cast<uint16_t *>(out)[at] = Elem<DT>::narrow(v);
    }
}

// ---------------------------------------------------------------- launches

template <int DT, bool TR> hipError_t shrink_go(const LoraParams &p, hipStream_t stream)
{
    const int64_t tiles = (p.T + kShrinkRows - 1) / kShrinkRows + (p.T < p.L ? p.T : p.L);
    const dim3 grid((unsigned)(tiles * p.splits)), block(kShrinkWaves * kWave);
    if (p.R <= 16)
        hipLaunchKernelGGL((shrink_kernel<DT, TR, 1>), grid, block, 0, stream, p);
    else if (p.R <= 32)
        hipLaunchKernelGGL((shrink_kernel<DT, TR, 2>), grid, block, 0, stream, p);
    else if (p.R <= 64)
        hipLaunchKernelGGL((shrink_kernel<DT, TR, 4>), grid, block, 0, stream, p);
    else if (p.R <= 128)
        hipLaunchKernelGGL((shrink_kernel<DT, TR, 8>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((shrink_kernel<DT, TR, 16>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int DT, bool TR> hipError_t expand_go(const LoraParams &p, hipStream_t stream)
{
    const int rows = TR ? kExpandRowsT : kExpandRows;
    const int cols = 4 * (TR ? 128 : 64);
    const int64_t tiles = (p.T + rows - 1) / rows + (p.T < p.L ? p.T : p.L);
    const int col_tiles = (p.C + cols - 1) / cols;
    const dim3 grid((unsigned)(tiles * col_tiles));
    if (p.R <= 16)
        hipLaunchKernelGGL((expand_kernel<DT, TR, true>), grid, dim3(256), 0, stream, p, col_tiles);
    else
        hipLaunchKernelGGL((expand_kernel<DT, TR, false>), grid, dim3(256), 0, stream, p,
                           col_tiles);
    return hipGetLastError();
}

template <int DT> hipError_t grad_go(const GradParams &p, hipStream_t stream)
{
    const int64_t items = p.l.L + p.l.T / p.chunk;
    const int rg = p.R <= 16 ? 1 : 2;
    const int64_t rank_tiles = (p.R + rg * 16 - 1) / (rg * 16);
    const dim3 grid((unsigned)(items * (p.col_tiles_a + p.col_tiles_b) * rank_tiles));
    if (rg == 1)
        hipLaunchKernelGGL((grad_kernel<DT, 1>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((grad_kernel<DT, 2>), grid, dim3(256), 0, stream, p);
    if (p.l.T <= p.chunk)
        return hipGetLastError();
    const int blocks = 64;
    hipLaunchKernelGGL((grad_join_kernel<DT>), dim3((unsigned)(p.l.L * blocks)), dim3(256), 0,
                       stream, p, blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t lora_shrink_launch(const LoraParams &p, int dtype, bool transposed, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    if (dtype == kBf16)
        return transposed ? shrink_go<kBf16, true>(p, stream) : shrink_go<kBf16, false>(p, stream);
    return transposed ? shrink_go<kFp16, true>(p, stream) : shrink_go<kFp16, false>(p, stream);
}

hipError_t lora_expand_launch(const LoraParams &p, int dtype, bool transposed, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    if (dtype == kBf16)
        return transposed ? expand_go<kBf16, true>(p, stream) : expand_go<kBf16, false>(p, stream);
    return transposed ? expand_go<kFp16, true>(p, stream) : expand_go<kFp16, false>(p, stream);
}

hipError_t lora_grad_launch(const GradParams &p, int dtype, hipStream_t stream)
{
    return dtype == kBf16 ? grad_go<kBf16>(p, stream) : grad_go<kFp16>(p, stream);
}

}  // namespace moegg
