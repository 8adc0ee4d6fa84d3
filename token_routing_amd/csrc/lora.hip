// Low-rank adapters of many requests beside a shared projection, gfx950.
//
//   forward   h[p] = x[src(p)] A_a^T                      (shrink)
//             y[src(p)] = base[src(p)] + s_a h[p] B_a^T   (expand)
//   backward  dh[p] = s_a dy[src(p)] B_a                  (shrink, B transposed)
//             dx[src(p)] = base[src(p)] + dh[p] A_a       (expand, A transposed)
//             dA_a = sum_p dh[p]^T x[src(p)], dB_a = s_a sum_p dy[src(p)]^T h[p]  (grad)
//
// for sorted position p of adapter a.  With ranks up to 64 against rows of
// thousands of columns every one of these is bound by moving x, y and dy, not
// by its matrix instructions (16 x 16 x 32, fp32 accumulators).  So no tile is
// staged for reuse between waves: a wave loads what it multiplies, 8 reduction
// elements (16 contiguous bytes) a lane, and LDS only moves values between the
// lanes of a wave where the layout of a fragment would waste cache lookups.
// Above rank 64 that costs: shrink's 16-row tiles read 8 (rank 128) to 16 times
// (256) their rows' bytes in weights from the caches, and grad reads x and dy
// once for every 32 ranks.
//
// Operands whose reduction runs along a strided index (B in dh, A in dx, x and
// dy in the gradients) are loaded as 8 rows of up to 8 contiguous elements a
// lane and transposed in registers, two 16-bit halves per byte permute.  The
// reduction order inside an instruction is free as long as both operands
// agree, and so is the assignment of output columns to lanes.
//
// h and dh stay in fp32 between the kernels.  Where one enters a matrix
// instruction it goes as the sum of 16-bit values, each the rounded rest of the
// ones before, at as many matrix instructions, of which there are few.  Two in
// fp16 keep 22 bits of mantissa, three in bf16 hold an fp32 value whole.  Two in
// bf16 kept 16 bits, which showed in fp32 gradients (4096 rows, rank 32: off by
// 2.5e-6 in norm, 1.8e-7 with three) and in outputs where base and the adapter
// cancel; the third part costs nothing in the gradients (53.8 us the call with
// either), 1 us of 139 in expand at rank 64 into 28672 columns, 2 of 59 at rank
// 128 and 4 of 71 at rank 256.  With ranks up to 16 two parts share one
// instruction of expand: its 32 reduction elements hold 16 of each.  fp16 parts
// are scaled by a power of two first, so that values past the type's range
// survive.
//
// Rows go by tiles inside one adapter's segment; each wave finds its tile by
// a scan of m_sizes in registers (64 segments a step), so no launch depends
// on the host knowing the sizes.
#include <type_traits>

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

// Inclusive scan over the wave by data-parallel moves inside the registers (a
// lane shift through LDS costs ten times as much, and every launch waits for
// its scans first).  add(x, 0) has to be x.
template <class Add> __device__ __forceinline__ uint32_t wave_scan(uint32_t v, Add add)
{
    v = add(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // row_shr:1
    v = add(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));  // row_shr:2
    v = add(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));  // row_shr:4
    v = add(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));  // row_shr:8
    v = add(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // row_bcast:15
    v = add(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return v;
}

__device__ __forceinline__ int lane_of(uint32_t v, int lane)
{
    return __builtin_amdgcn_readlane((int)v, lane);
}

// The tile `want` of all segments' tiles of `per` rows (empty segments have
// `empty` tiles); false past the last one, with its distance from it in t.index
// and the segments' rows together in t.p0.  By adapter with by_adapter: the
// segment of adapter `want`.  All lanes of the wave call it.  Row sums
// saturate at S, so that bad sizes cannot wrap around.
__device__ __forceinline__ bool find_tile(const int32_t *m_sizes, int L, uint32_t S, int want,
                                          int per, int empty, bool by_adapter, Tile &t)
{
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t row0 = 0;
    int tile0 = 0, slot0 = 0;
    for (int c = 0; c < L; c += kWave) {
        const int a = c + lane;
        const int raw = m_sizes[min(a, L - 1)];
        const uint32_t v = a < L ? min((uint32_t)max(raw, 0), S) : 0;
        const uint32_t end = min(
            wave_scan(v, [S](uint32_t x, uint32_t y) { return min(x + y, S); }) + row0, S);
        // The row before a segment: the lane below's end (the first lane's is row0).
        uint32_t start = __builtin_amdgcn_update_dpp(row0, end, 0x138, 0xf, 0xf, false);  // wave_shr:1
        const int m = (int)(end - start);
        const int n = m > 0 ? (m - 1) / per + 1 : (a < L ? empty : 0);
        const auto sum = [](uint32_t x, uint32_t y) { return x + y; };
        const int tiles = (int)wave_scan(n, sum);
        const int slots = (int)wave_scan(n > 1 ? n : 0, sum);
        const uint64_t hit =
            __ballot(by_adapter ? a == want : a < L && tile0 + tiles > want);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            t.a = c + l;
            t.m = lane_of(m, l);
            t.index = by_adapter ? 0 : want - (tile0 + lane_of(tiles - n, l));
            t.p0 = lane_of(start, l) + t.index * per;
            t.rows = min(per, t.m - t.index * per);
            t.slot = slot0 + lane_of(slots, l) - (t.m > per ? (t.m - 1) / per + 1 : 0);
            return true;
        }
        row0 = lane_of(end, kWave - 1);
        tile0 += lane_of(tiles, kWave - 1);
        slot0 += lane_of(slots, kWave - 1);
    }
    t.index = want - tile0;
    t.p0 = (int)row0;
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

// 8 elements that are known to lie inside their array.
__device__ __forceinline__ u32x4_t load8_in(const uint16_t *p)
{
    typedef Pack16<kBf16>::vec_t vec_t;
    return __builtin_bit_cast(u32x4_t, *reinterpret_cast<const vec_t *>(p));
}

// The same with the nontemporal hint: the line is not kept for a later read.
__device__ __forceinline__ u32x4_t load8_stream(const uint16_t *p)
{
    typedef Pack16<kBf16>::vec_t vec_t;
    return __builtin_bit_cast(
        u32x4_t, __builtin_nontemporal_load(reinterpret_cast<const vec_t *>(p)));
}

// Elements [at, at + 8) of an array of n >= 8 elements, zero past its end:
// the load is moved back inside and its elements shifted down.
__device__ __forceinline__ u32x4_t load8_end(const uint16_t *p, int64_t at, int64_t n)
{
    typedef unsigned long long u64x2_t __attribute__((ext_vector_type(2)));
    const int64_t start = min(at, n - 8);
    const u64x2_t v = __builtin_bit_cast(u64x2_t, load8_in(p + start));
    const int64_t by = at - start;
    const int s = ((int)by & 3) * 16;
    const unsigned long long low = by >= 4 ? v[1] : v[0], high = by >= 4 ? 0 : v[1];
    u64x2_t r;
    r[0] = by >= 8 ? 0 : low >> s | (s ? high << (64 - s) : 0);
    r[1] = by >= 8 ? 0 : high >> s;
    return __builtin_bit_cast(u32x4_t, r);
}

// W elements that are known to lie inside their array, as packed pairs.
template <int W>
__device__ __forceinline__ void load_pairs(uint32_t (&d)[W < 2 ? 1 : W / 2], const uint16_t *p)
{
    typedef uint16_t vec_t __attribute__((ext_vector_type(W < 2 ? 2 : W), aligned(2)));
    if constexpr (W == 1) {
        d[0] = *p;
    } else {
        const vec_t v = *reinterpret_cast<const vec_t *>(p);
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
            d[i] = (uint32_t)v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
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

// v as the sum of PARTS 16-bit values, each the rounded rest of the ones before.
// A value that is not finite has no rest.  Two parts hold 16 bits of mantissa in
// bf16 and 22 in fp16, three all 24 of an fp32 value in bf16.
template <int DT, int PARTS>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4_t (&part)[PARTS])
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        float r[2] = {v[2 * d], v[2 * d + 1]};
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            float h[2];
            if constexpr (DT == kBf16) {
                const uint32_t both = pack_bf16x2(r[0], r[1]);
                part[p][d] = both;
                h[0] = __builtin_bit_cast(float, both << 16);
                h[1] = __builtin_bit_cast(float, both & 0xffff0000u);
            } else {
                const uint32_t a = Elem<kFp16>::narrow(r[0]), b = Elem<kFp16>::narrow(r[1]);
                part[p][d] = a | b << 16;
                h[0] = Elem<kFp16>::widen((uint16_t)a);
                h[1] = Elem<kFp16>::widen((uint16_t)b);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                r[i] = p > 0 || fabsf(h[i]) < __builtin_huge_valf() ? r[i] - h[i] : 0.0f;
        }
    }
}

// h[p][col .. col + 8), the splits' partial sums added in order, 0 from n on.
// May read up to 8 values past the row (h has that much room behind it).
__device__ __forceinline__ void load_h(float (&v)[8], const float *h, int64_t p, int R, int col,
                                       int n, int splits, int64_t split_stride)
{
    const float *q = h + p * R + (col < n ? col : 0);
    f32x4_t a = *reinterpret_cast<const f32x4u_t *>(q);
    f32x4_t b = *reinterpret_cast<const f32x4u_t *>(q + 4);
    for (int s = 1; s < splits; s += 2) {
        f32x4_t c[2], d[2];  // two splits' loads at once, the last one's again past the end
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float *const r = q + min(s + u, splits - 1) * split_stride;
            c[u] = *reinterpret_cast<const f32x4u_t *>(r);
            d[u] = *reinterpret_cast<const f32x4u_t *>(r + 4);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (s + u < splits) {
                a += c[u];
                b += d[u];
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = col + i < n ? a[i] : 0.0f;
        v[4 + i] = col + 4 + i < n ? b[i] : 0.0f;
    }
}

// ---------------------------------------------------------------- shrink

// h[p, r] = factor * sum_c in[src(p), c] * w(r, c) for a tile of RT * 16 rows:
// w(r, c) = W[r][c] (W [R, C], forward) or W[c][r] (W [C, R], TR).  A
// workgroup of 8 waves takes 1 / splits of the reduction, each wave an equal
// run of it, and adds the waves' sums through LDS in wave order.  Each split
// stores a copy of its own.  RF: 16-row blocks of ranks.
//
// Loaded in the layout of a fragment, 16 neighbouring lanes on 16 rows, every
// 16 bytes would be a cache lookup of their own, and the lookups the bound;
// rows are loaded 64 bytes at a time instead and reach their lanes through
// LDS.  RT > 1 uses the weights' fragments for several blocks of rows.
//
// The loads of U whole 32-column steps are issued together, without branches:
// lanes past the tile's rows load its first row again and lanes past the rank
// another row of weights, since a matrix instruction keeps them in outputs of
// their own, which are not stored.  EDGE: columns that are no whole steps, or
// ranks that are no whole pieces of 4 or of a lane (TR).  Code is kept short
// on purpose: a wave runs most of it once, and fetching it cost more than the
// loads when every guarded element had its own branch.
//
// 4096 rows of 4096 columns: 16.7 us at rank 64, 13.0 us transposed at rank 32
// (33 MB of rows, 2.0 and 2.6 TB/s): one or two round trips to memory after the
// tile, rank and row numbers, and the waves' sums behind them.
constexpr int kShrinkWaves = 8;

template <int DT, bool TR, int RF, int RT, bool EDGE>
__global__ __launch_bounds__(kShrinkWaves *kWave, RF <= 8 ? 4 : 2) void shrink_kernel(LoraParams a)
{
    // With TR a lane holds ranks m * RF + j, one piece of a row of weights;
    // with EDGE ranks f * 16 + m, one element of a row at a time.
    constexpr bool PIECES = TR && !EDGE;
    constexpr int W = PIECES ? RF : 1;
    constexpr int D = W < 2 ? 1 : W / 2;
    constexpr int Q = TR ? (PIECES ? 1 : RF) : 1;  // loads of a row of weights (TR)
    constexpr int U = TR && EDGE ? (RF <= 2 ? 2 : 1) : RF <= 2 ? 4 : RF <= 8 ? 2 : 1;
    constexpr int kBlocks = RT * RF, kTurn = kBlocks < kShrinkWaves ? kBlocks : kShrinkWaves;
    __shared__ f32x4_t s_acc[kShrinkWaves][kTurn][kWave];
    check_sizes(a.m_sizes, a.ranks, a.L, a.T, a.R, a.err);
    const int split = blockIdx.x % a.splits;
    Tile tile;
    if (!find_tile(a.m_sizes, a.L, (uint32_t)a.T, blockIdx.x / a.splits, RT * 16, 0, false, tile))
        return;
    const int rank = rank_of(a.ranks, tile.a, a.R);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int m = lane & 15, g = lane >> 4;

    // Rows are loaded four lanes to a row, 64 bytes of it, and change lanes
    // through LDS: lane 4 r + q loads piece q of row r, lane 16 g + m needs
    // piece g of row m.  The pieces of a row are exchanged so that neither
    // access has two lanes on one bank.
    const int rl = lane >> 2, ql = lane & 3;
    const int put_at = rl * 4 + (ql ^ ((rl >> 1) & 3)), get_at = m * 4 + (g ^ ((m >> 1) & 3));
    const uint16_t *row[RT];
    uint32_t bad_rows = 0;  // bit t: the lane's row of block t has a bad gather entry
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int64_t src = source_row(a, tile.p0 + (t * 16 + rl < tile.rows ? t * 16 + rl : 0));
        bad_rows |= (uint32_t)(src < 0) << t;
        row[t] = a.in + (src < 0 ? 0 : src) * a.ld_in;
    }
    const uint16_t *const w = a.w + (int64_t)tile.a * a.R * a.C;

    f32x4_t acc[RT][RF];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int f = 0; f < RF; ++f)
            acc[t][f] = f32x4_t{};
    const int whole = a.C / 32, steps = EDGE ? (a.C + 31) / 32 : whole;
    const int parts = a.splits * kShrinkWaves;
    const int part = split * kShrinkWaves + wave;
    const int s0 = (int)((int64_t)steps * part / parts);
    const int s1 = (int)((int64_t)steps * (part + 1) / parts);
    const int full = EDGE ? min(s1, whole) : s1;
    if (rank > 0) {
        const uint16_t *wrow[TR ? Q : RF];
#pragma unroll
        for (int f = 0; f < (TR ? Q : RF); ++f) {
            if constexpr (PIECES)
                wrow[f] = w + min(m * W, a.R - W);
            else if constexpr (TR)
                wrow[f] = w + min(f * 16 + m, a.R - 1);
            else
                wrow[f] = w + (int64_t)min(f * 16 + rl, rank - 1) * a.C;
        }
        u32x4_t *const stage = reinterpret_cast<u32x4_t *>(&s_acc[wave][0][0]);
        // One step from its loaded rows: x into LDS and back, then the weights,
        // kTurn blocks (the room a wave has) at a time.
        auto step = [&](const u32x4_t (&x)[RT], auto &&weights) {
            u32x4_t xf[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t)
                stage[t * kWave + put_at] = x[t];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int t = 0; t < RT; ++t)
                xf[t] = stage[t * kWave + get_at];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int f0 = 0; f0 < RF; f0 += kTurn) {
                if constexpr (!TR) {
#pragma unroll
                    for (int f = 0; f < kTurn && f0 + f < RF; ++f)
                        stage[f * kWave + put_at] = weights(f0 + f);
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
#pragma unroll
                for (int f = 0; f < kTurn && f0 + f < RF; ++f) {
                    const u32x4_t b = TR ? weights(f0 + f) : stage[f * kWave + get_at];
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[t][f0 + f] = mfma<DT>(b, xf[t], acc[t][f0 + f]);
                }
                if constexpr (!TR) {
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
            }
        };
        for (int s = s0; s < full; s += U) {
            u32x4_t x[U][RT], v[TR ? 1 : U][TR ? 1 : RF];
            uint32_t q[TR ? U : 1][Q][8][D];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c0 = min(s + u, full - 1) * 32;
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    x[u][t] = load8_in(row[t] + c0 + ql * 8);
                if constexpr (!TR) {
#pragma unroll
                    for (int f = 0; f < RF; ++f)
                        v[u][f] = load8_in(wrow[f] + c0 + ql * 8);
                } else {
#pragma unroll
                    for (int f = 0; f < Q; ++f)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            load_pairs<W>(q[u][f][e], wrow[f] + (int64_t)(c0 + g * 8 + e) * a.R);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < full)
                    step(x[u], [&](int f) {
                        return TR ? column<W>(q[TR ? u : 0][PIECES ? 0 : TR ? f : 0],
                                              PIECES ? f : 0)
                                  : v[TR ? 0 : u][TR ? 0 : f];
                    });
        }
        if constexpr (EDGE) {
            if (s1 > whole && s0 < s1) {  // the last, partial step
                const int c0 = whole * 32;
                u32x4_t x[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    x[t] = load8_end(row[t], c0 + ql * 8, a.C);
                step(x, [&](int f) {
                    if constexpr (TR) {
                        uint32_t e8[8][1];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int c = c0 + g * 8 + e;
                            load_pairs<1>(e8[e], wrow[f] + (int64_t)min(c, a.C - 1) * a.R);
                            e8[e][0] = c < a.C ? e8[e][0] : 0;
                        }
                        return column<1>(e8, 0);
                    } else {
                        return load8_end(wrow[f], c0 + ql * 8, a.C);
                    }
                });
            }
        }
    }
    // Every wave adds, in wave order, and stores the blocks of sums that are its
    // share: 8 blocks at a time, one a wave.
    const float factor = a.scale_shrink && a.scales ? a.scales[tile.a] : 1.0f;
    // The lane that loaded row m knows whether it was bad.
    bad_rows = __shfl(bad_rows, m * 4, kWave);
#pragma unroll
    for (int turn = 0; turn < kBlocks; turn += kTurn) {
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kTurn; ++b)
            s_acc[wave][b][lane] = acc[(turn + b) / RF][(turn + b) % RF];
        __syncthreads();
        if (wave >= kTurn)
            continue;
        f32x4_t sum = s_acc[0][wave][lane];
#pragma unroll
        for (int i = 1; i < kShrinkWaves; ++i)
            sum += s_acc[i][wave][lane];
        // A block's outputs: row t * 16 + m, and ranks f * 16 + 4 g + i or, with
        // PIECES, (4 g + i) * RF + f.
        const int t = (turn + wave) / RF, f = (turn + wave) % RF;
        const int p = tile.p0 + t * 16 + m;
        if (t * 16 + m >= tile.rows)
            continue;
        const bool bad = bad_rows >> t & 1;
        float *const h = a.h + split * a.split_stride + (int64_t)p * a.R;
        f32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = PIECES ? (4 * g + i) * RF + f : f * 16 + 4 * g + i;
            v[i] = r < rank && !bad ? factor * sum[i] : 0.0f;
            if ((EDGE || PIECES) && r < a.R)
                h[r] = v[i];
        }
        if (!EDGE && !PIECES && f * 16 + 4 * g < a.R)
            *reinterpret_cast<f32x4u_t *>(h + f * 16 + 4 * g) = v;
    }
}

// ---------------------------------------------------------------- expand

// out[src(p), c] = base[src(p), c] + factor * sum_r h[p, r] * w(r, c), w(r, c)
// = W[c][r] (W [C, R], forward) or W[r][c] (W [R, C], TR).
//
// A workgroup takes up to RT * 16 rows of one adapter and a run of columns, its
// waves 64 columns each at a time; rows past the tile's repeat its last one and
// are not stored.  h is split into its parts once and kept in LDS as
// fragments (NS steps of 32 ranks).  A wave's pass: the weights' fragments (each
// used for all rows), the matrix instructions, and the sums through a strip of
// LDS into row order, so that base is read and out written in whole 128-byte
// lines: straight from the accumulators' layout every 16 bytes of a line would
// be looked up apart, which took 1.7 times as long.  The next pass's weights
// are issued after this one's matrix instructions and its base as this one's is
// used, in the order in which they are waited for.
//
// 4096 rows, 8 adapters of rank up to 64, 28672 columns: 120 us, 3.9 TB/s of
// base and out, of which 9 us pass before the first pass; HBM is the bound
// inside the passes.  64 rows over 32 adapters of rank 16, 4096 columns: 5.8 us,
// four dependent loads long.
//
// SMALL: ranks up to 16, two parts of h in one instruction.  EDGE: columns that
// are no whole passes (the last one goes by single elements) or ranks that are
// no whole pieces of 8.  expand_places: workgroups a compute unit, by registers, and
// above rank 128 with 64-row tiles by shared memory (116 KB a workgroup).
// Registers spilled to scratch, of 256: 30 to 46 in the 64-row dX at ranks 65 to
// 128 (35.3 us at rank 128, 4096 rows of 4096 columns, where the forward takes
// 29.7); 15 at most in sixteen forms of other ranks and tiles.
constexpr int expand_places(bool TR, int NS, int RT)
{
    return RT == 1 ? (NS <= 2 ? 4 : NS == 8 && TR ? 2 : 3)
           : NS == 8                          ? 1
           : NS == 1 || (NS == 2 && !TR)      ? 3
                                              : 2;
}

// Rows at no sorted position below `sum` get base's row in columns [c0, c1):
// workgroup `index` of `workgroups` takes an even share of the rows (without a
// gather index those behind the sum), marks in `mark` which of them are routed,
// and copies the others.
__device__ __forceinline__ void copy_unrouted(const LoraParams &a, int sum, int index,
                                              int workgroups, int c0, int c1, uint32_t *mark,
                                              int words)
{
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int first = a.gather ? 0 : sum;
    const int per = ((int)a.T - first + workgroups - 1) / workgroups;
    const int lo = first + index * per, hi = min((int)a.T, lo + per);
    for (int r0 = lo; r0 < hi; r0 += words * 32) {
        const int n = min(words * 32, hi - r0);
        if (a.gather) {
            for (int i = threadIdx.x; i < (n + 31) / 32; i += 256)
                mark[i] = 0;
            __syncthreads();
            for (int p = threadIdx.x; p < sum; p += 256) {
                const uint32_t d = (uint32_t)a.gather[p] - (uint32_t)r0;
                if (d < (uint32_t)n)
                    atomicOr(&mark[d / 32], 1u << d % 32);
            }
            __syncthreads();
        }
        for (int i = wave; i < n; i += 4) {
            if (a.gather && (mark[i / 32] >> i % 32 & 1))
                continue;
            const uint16_t *const from = a.base + (int64_t)(r0 + i) * a.ld_base;
            uint16_t *const to = a.out + (int64_t)(r0 + i) * a.ld_out;
            for (int c = c0 + lane * 8; c < c1; c += kWave * 8) {
                if (c + 8 <= c1) {
                    *reinterpret_cast<Pack16<kBf16>::vec_t *>(to + c) =
                        *reinterpret_cast<const Pack16<kBf16>::vec_t *>(from + c);
                } else {
                    for (int e = c; e < c1; ++e)
                        to[e] = from[e];
                }
            }
        }
        __syncthreads();
    }
}

template <int DT, bool TR, int NS, bool SMALL, int RT, bool EDGE>
__global__ __launch_bounds__(256, expand_places(TR, NS, RT)) void
expand_kernel(LoraParams a, int groups, int group_cols)
{
    constexpr int F = 4;
    constexpr int kCols = F * 16;
    constexpr int kRows = RT * 16;
    constexpr int kPad = kCols + 4;
    constexpr bool STEPWISE = NS > 2;
    constexpr int kParts = DT == kBf16 ? 3 : 2;
    constexpr int kFragments = SMALL ? (kParts + 1) / 2 : kParts;  // of h, a step and block
    __shared__ u32x4_t s_h[NS][RT][kFragments][kWave];
    __shared__ __attribute__((aligned(16))) float s_out[4][16][kPad];
    __shared__ int s_src[kRows];
    __shared__ float s_factor[kRows];
    const int group = blockIdx.x % groups;
    Tile tile;
    if (!find_tile(a.m_sizes, a.L, (uint32_t)a.T, blockIdx.x / groups, kRows, 0, false, tile)) {
        // The grid holds ceil(T / kRows) + min(T, L) tiles, more than the sum of
        // the adapters' when that is below T: at least one workgroup a column
        // group gets here.  Each reads all of the gather index, so 512 at most.
        if (a.copy_unrouted && tile.p0 < a.T) {
            const int tiles = blockIdx.x / groups - tile.index;
            const int most = groups < 512 ? 512 / groups : 1;
            const int workgroups = min((int)(gridDim.x / groups) - tiles, most);
            if (tile.index < workgroups)
                copy_unrouted(a, tile.p0, tile.index, workgroups, group * group_cols,
                              min(a.C, (group + 1) * group_cols),
                              reinterpret_cast<uint32_t *>(s_out), sizeof(s_out) / 4);
        }
        return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int m = lane & 15, g = lane >> 4;
    const int rank = rank_of(a.ranks, tile.a, a.R);
    const int rg = SMALL ? (g & 1) * 8 : g * 8;  // this lane's ranks of a step

    // In row order a lane holds 8 columns of rows lane / 8 and lane / 8 + 8 of
    // a block.  A bad gather entry (shrink reports it) has no row.
    const int row_lane = lane >> 3, col_lane = (lane & 7) * 8;
    int src[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = t * 16 + i * 8 + row_lane;
            const int p = tile.p0 + min(r, tile.rows - 1);
            const int x = a.gather ? a.gather[p] : p;
            src[t][i] = r < tile.rows && x >= 0 && x < a.T ? x : -1;
        }
    const int c_end = min(a.C, (group + 1) * group_cols);
    const int c_begin = group * group_cols + wave * kCols;
    u32x4_t old[RT][2];
    auto load_base = [&](int t, int c0) {
        const int c = EDGE ? min(c0 + col_lane, a.C - 8) : c0 + col_lane;
        const uint16_t *const q0 = a.base + (int64_t)max(src[t][0], 0) * a.ld_base + c;
        const uint16_t *const q1 = a.base + (int64_t)max(src[t][1], 0) * a.ld_base + c;
        // The empty statements keep the compiler from making one pair of loads
        // of the two, without the hint.
        if (a.stream_base) {
            asm volatile("");
            old[t][0] = load8_stream(q0);
            old[t][1] = load8_stream(q1);
            asm volatile("");
        } else {
            old[t][0] = load8_in(q0);
            old[t][1] = load8_in(q1);
        }
    };

    // A step's weights of the lane, as loaded: forward 4 fragments, TR 8 rows
    // of 4 columns.  Every address lies inside the adapter's weights.
    const uint16_t *const w = a.w + (int64_t)tile.a * a.R * a.C;
    uint32_t raw[STEPWISE ? 2 : NS][8][2];
    auto load_weights = [&](uint32_t (&v)[8][2], int s, int c0) {
        const int r0 = s * 32 + rg;
        if constexpr (TR) {
            // The last lanes' columns are moved inside the row.
            const int c = EDGE ? min(c0 + m * 4, a.C - 4) : c0 + m * 4;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                load_pairs<4>(v[e], w + (int64_t)min(r0 + e, a.R - 1) * a.C + c);
        } else {
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int c = c0 + f * 16 + m;
                const int64_t at =
                    (int64_t)(EDGE ? min(c, a.C - 1) : c) * a.R + (r0 < a.R ? r0 : 0);
                const u32x4_t b = EDGE ? load8_end(w, at, (int64_t)a.C * a.R) : load8_in(w + at);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[(4 * f + i) / 2][(4 * f + i) % 2] = b[i];
            }
        }
    };

    // Weights first, then base, then h: all in flight together, and base does
    // not wait for the conversion of h.  (Above rank 64 the registers hold
    // only one of them at a time.)
    auto load_first = [&] {
        if (c_begin >= c_end)
            return;
#pragma unroll
        for (int s = 0; s < (STEPWISE ? 1 : NS); ++s)
            load_weights(raw[s], s, c_begin);
#pragma unroll
        for (int t = 0; t < RT; ++t)
            load_base(t, c_begin);
    };
    if constexpr (!STEPWISE)
        load_first();
    if (wave < RT) {
        const int t = wave * 16 + m;
        const int p = tile.p0 + min(t, tile.rows - 1);
        // Rank 0 is no adapter, whatever its scale holds.
        float factor = !a.scale_shrink && a.scales && rank > 0 ? a.scales[tile.a] : 1.0f;
        float v[NS][8];
#pragma unroll
        for (int s = 0; s < NS; ++s)
            load_h(v[s], a.h, p, a.R, s * 32 + rg, rank, a.splits, a.split_stride);
        // The summed h for the caller, by the first column group.
        if (a.h_out && group == 0 && t < tile.rows && (!SMALL || g < 2))
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int r = s * 32 + rg;
                float *const q = a.h_out + (int64_t)p * a.R + r;
                if (!EDGE && r < a.R) {
                    *reinterpret_cast<f32x4u_t *>(q) = f32x4_t{v[s][0], v[s][1], v[s][2], v[s][3]};
                    *reinterpret_cast<f32x4u_t *>(q + 4) =
                        f32x4_t{v[s][4], v[s][5], v[s][6], v[s][7]};
                } else if (EDGE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (r + i < a.R)
                            q[i] = v[s][i];
                }
            }
        if constexpr (DT == kFp16) {
            float top = 0.0f;
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = fmaxf(top, fabsf(v[s][i]));
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            const float fit = fit_scale(top);
            factor *= inverse_scale(fit);
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[s][i] *= fit;
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            u32x4_t part[kParts];
            split8<DT>(v[s], part);
#pragma unroll
            for (int i = 0; i < kFragments; ++i) {
                u32x4_t f = part[SMALL ? 2 * i : i];
                if constexpr (SMALL)
                    if (g >= 2)
                        f = 2 * i + 1 < kParts ? part[min(2 * i + 1, kParts - 1)] : u32x4_t{};
                s_h[s][wave][i][lane] = f;
            }
        }
        if (g == 0)
            s_factor[t] = factor;
        if constexpr (EDGE) {
            const int x = a.gather ? a.gather[p] : p;
            if (g == 0)
                s_src[t] = t < tile.rows && x >= 0 && x < a.T ? x : -1;
        }
    }
    if constexpr (STEPWISE)
        load_first();
    __syncthreads();
    if (c_begin >= c_end || (rank == 0 && a.base == a.out))
        return;

    // One pass.  MORE: another one follows, fixed at compile time, since a load
    // under a branch makes every later wait count as if it had not been issued.
    auto pass = [&](int c0, auto more_c) {
        constexpr bool MORE = decltype(more_c)::value;
        // Fragments of a step; ranks at or past the rank may hold anything.
        auto fragments = [&](u32x4_t (&wf)[F], const uint32_t (&v)[8][2], int s) {
            const int left = rank - (s * 32 + rg);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                if constexpr (TR)
                    wf[f] = column<4>(v, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (!TR)
                        wf[f][i] = v[(4 * f + i) / 2][(4 * f + i) % 2];
                    wf[f][i] &= left > 2 * i + 1 ? ~0u : left > 2 * i ? 0xffffu : 0u;
                }
            }
        };
        auto multiply = [&](f32x4_t (&acc)[F], const u32x4_t (&wf)[F], int s, int t) {
#pragma unroll
            for (int part = 0; part < kFragments; ++part) {
                const u32x4_t h = s_h[s][t][part][lane];
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc[f] = mfma<DT>(wf[f], h, acc[f]);
            }
        };
        // Up to rank 64 a pass's weights are all in registers, and one block's
        // sums at a time; above, all blocks' sums, and two steps' weights.
        u32x4_t wf[STEPWISE ? 1 : NS][F];
        f32x4_t acc_all[STEPWISE ? RT : 1][F];
        if constexpr (STEPWISE) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc_all[t][f] = f32x4_t{};
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                if (s + 1 < NS)
                    load_weights(raw[(s + 1) & 1], s + 1, c0);
                fragments(wf[0], raw[s & 1], s);
                if (MORE && s + 1 == NS)
                    load_weights(raw[0], 0, c0 + 4 * kCols);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    multiply(acc_all[t], wf[0], s, t);
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; ++s)
                fragments(wf[s], raw[s], s);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            f32x4_t acc[F];
            if constexpr (STEPWISE) {
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc[f] = acc_all[t][f];
            } else {
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc[f] = f32x4_t{};
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    multiply(acc, wf[s], s, t);
                if (MORE && t == RT - 1)
#pragma unroll
                    for (int s = 0; s < NS; ++s)
                        load_weights(raw[s], s, c0 + 4 * kCols);
            }
            // A lane holds row m, columns f * 16 + 4 g + i (TR: (4 g + i) * 4 + f).
            const bool inside = !EDGE || MORE || c0 + kCols <= a.C;
            if (!TR || inside) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4_t v =
                        TR ? f32x4_t{acc[0][i], acc[1][i], acc[2][i], acc[3][i]} : acc[i];
                    *reinterpret_cast<f32x4_t *>(
                        &s_out[wave][m][TR ? (4 * g + i) * 4 : i * 16 + 4 * g]) = v;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = min(c0 + (4 * g + i) * 4, a.C - 4) - c0;
#pragma unroll
                    for (int f = 0; f < F; ++f)
                        if (c + f >= 0)
                            s_out[wave][m][c + f] = acc[f][i];
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (inside) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = i * 8 + row_lane;
                    const f32x4_t *const d =
                        reinterpret_cast<const f32x4_t *>(&s_out[wave][r][col_lane]);
                    const f32x4_t d0 = d[0], d1 = d[1];
                    const float k = s_factor[t * 16 + r];
                    float y[8];
                    widen_all<DT>(y, __builtin_bit_cast(typename Pack16<DT>::vec_t, old[t][i]));
                    typename Pack16<DT>::vec_t out;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] += k * d0[e];
                        y[4 + e] += k * d1[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        out[e] = Elem<DT>::narrow(y[e]);
                    if (src[t][i] >= 0)
                        __builtin_nontemporal_store(
                            out, reinterpret_cast<typename Pack16<DT>::vec_t *>(
                                     a.out + (int64_t)src[t][i] * a.ld_out + c0 + col_lane));
                }
                if constexpr (MORE)
                    load_base(t, c0 + 4 * kCols);
            } else {
                // A column a lane, 8 rows at once.
                const int c = c0 + lane;
                for (int r0 = 0; r0 < 16; r0 += 8) {
                    int64_t row[8];
                    uint16_t was[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        row[u] = s_src[t * 16 + r0 + u];
                        was[u] = a.base[max(row[u], (int64_t)0) * a.ld_base + min(c, a.C - 1)];
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int r = r0 + u;
                        const float y = Elem<DT>::widen(was[u]) +
                                        s_factor[t * 16 + r] * s_out[wave][r][lane];
                        if (row[u] >= 0 && c < a.C)
                            a.out[row[u] * a.ld_out + c] = Elem<DT>::narrow(y);
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    };
    int c0 = c_begin;
    for (; c0 + 4 * kCols < c_end; c0 += 4 * kCols)
        pass(c0, std::true_type{});
    pass(c0, std::false_type{});
}

// ---------------------------------------------------------------- grad

// G[c, r] = factor * sum_p big[src(p), c] * small[p, r] over a chunk of one
// adapter's rows: dA (big = x, small = dh; stored [r][c]) in the first
// col_tiles_a column tiles, dB (big = dy, small = h; stored [c][r]) in the
// rest.  A workgroup of 4 waves takes 128 columns and RG * 16 ranks; the waves
// take turns at 32-row steps, leave their sums in LDS, and all of them add and
// store.  A segment of one chunk is finished here, the others leave fp32
// partials, cut evenly and in whole steps.
//
// A step is 8 rows of 16 bytes a lane, issued together; the rows' numbers are
// loaded a step ahead.  Rows past the chunk's end repeat its last row and are
// set to zero.  dh comes summed over shrink's splits.  4096 rows, 4 adapters of
// rank 32, K = N = 4096: 19.6 us for 67 MB of x and dy (3.4 TB/s), two waves a
// SIMD by registers and 1613 vector instructions a wave; every further 32 ranks
// read x and dy again: 29.7 us at rank 64, 61 us at 128.  Lanes past the last column load the row's last 8 elements and
// store only what is their own.
template <int DT, int RG>
__global__ __launch_bounds__(256) void grad_kernel(GradParams a)
{
    constexpr int kRanks = RG * 16;
    constexpr int kParts = DT == kBf16 ? 3 : 2;
    constexpr int kPad = 128 + 4;
    __shared__ __attribute__((aligned(16))) float s_sum[2][kRanks][kPad];
    const int rank_tiles = (a.R + kRanks - 1) / kRanks;
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
    const int rank = rank_of(a.l.ranks, tile.a, a.R);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int m = lane & 15, g = lane >> 4;
    const int r0 = rt * kRanks + m;

    const int chunks = tile.m > a.chunk ? (tile.m - 1) / a.chunk + 1 : 1;
    const int per = chunks > 1 ? ((tile.m + chunks - 1) / chunks + 31) / 32 * 32 : a.chunk;
    const int first = tile.p0 - tile.index * a.chunk;  // the segment's first position
    const int begin = first + min(tile.index * per, tile.m);
    const int end = first + min((tile.index + 1) * per, tile.m);

    f32x4_t acc[8][RG];
    float fit[RG];
#pragma unroll
    for (int q = 0; q < RG; ++q) {
        fit[q] = 1.0f;
#pragma unroll
        for (int f = 0; f < 8; ++f)
            acc[f][q] = f32x4_t{};
    }
    const int p_first = begin + wave * 32;
    if (p_first < end && rt * kRanks < rank) {
        const uint16_t *const big_c = big + min(ct * 128 + m * 8, C - 8);
        // Offsets of the lane's 8 rows of `small` in a step, ranks past the
        // rank clamped; the step's own start is the same for the wave.
        uint32_t small_at[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            small_at[e] = (uint32_t)((g * 8 + e) * a.R + min(r0, rank - 1));
        uint32_t block_at[RG];
#pragma unroll
        for (int q = 0; q < RG; ++q)
            block_at[q] = (uint32_t)(min(r0 + q * 16, rank - 1) - min(r0, rank - 1));
        auto rows_of = [&](int (&at)[8], int p) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                at[e] = min(p + g * 8 + e, end - 1);
            if (a.l.gather)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    at[e] = a.l.gather[at[e]];
        };
        auto load_small = [&](float (&v)[RG][8], int p) {
            const float *const s = small + (int64_t)p * a.R;
            if (p + 32 <= end) {
#pragma unroll
                for (int q = 0; q < RG; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[q][e] = s[small_at[e] + block_at[q]];
            } else {
#pragma unroll
                for (int q = 0; q < RG; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[q][e] = s[min(g * 8 + e, end - 1 - p) * a.R +
                                    min(r0 + q * 16, rank - 1)];
            }
        };
        if constexpr (DT == kFp16) {
            float top[RG] = {};
            for (int p = p_first; p < end; p += 128) {
                float v[RG][8];
                load_small(v, p);
#pragma unroll
                for (int q = 0; q < RG; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        top[q] = fmaxf(top[q], fabsf(v[q][e]));
            }
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                top[q] = fmaxf(top[q], __shfl_xor(top[q], 16, kWave));
                top[q] = fmaxf(top[q], __shfl_xor(top[q], 32, kWave));
                fit[q] = fit_scale(top[q]);
            }
        }
        int at[8];
        rows_of(at, p_first);
        for (int p = p_first; p < end; p += 128) {
            uint32_t rows[8][4];
            float h[RG][8];
            bool ok[8], odd = p + 32 > end;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ok[e] = (uint32_t)at[e] < (uint32_t)a.l.T;
                odd |= !ok[e];
                // ld is below 2^31: one multiply-add a row
                const uint16_t *const q =
                    big_c + (uint64_t)(ok[e] ? (uint32_t)at[e] : 0) * (uint32_t)ld;
                const u32x4_t v = load8_in(q);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rows[e][i] = v[i];
            }
            load_small(h, p);
            rows_of(at, p + 128);
            if (__ballot(odd))
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ok[e] = ok[e] && p + g * 8 + e < end;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        rows[e][i] = ok[e] ? rows[e][i] : 0;
#pragma unroll
                    for (int q = 0; q < RG; ++q)
                        h[q][e] = ok[e] ? h[q][e] : 0.0f;
                }
            u32x4_t part[RG][kParts];
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                // Columns of sums past the rank come from a clamped rank and are
                // set to zero when they are stored.
                if constexpr (DT == kFp16)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[q][e] *= fit[q];
                split8<DT>(h[q], part[q]);
            }
#pragma unroll
            for (int f = 0; f < 8; ++f) {
                const u32x4_t bf = column<8>(rows, f);
#pragma unroll
                for (int q = 0; q < RG; ++q)
#pragma unroll
                    for (int i = 0; i < kParts; ++i)
                        acc[f][q] = mfma<DT>(bf, part[q][i], acc[f][q]);
            }
        }
    }
    // A lane holds rank m of each block, columns (4 g + i) * 8 + f.  Waves 2 and
    // 3 leave their sums, waves 0 and 1 add theirs, and every thread adds the
    // two: (0 + 2) + (1 + 3).
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
        if (turn == (wave < 2))
#pragma unroll
            for (int q = 0; q < RG; ++q) {
                const float k = DT == kFp16 ? inverse_scale(fit[q]) : 1.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        f32x4_t *const d = reinterpret_cast<f32x4_t *>(
                            &s_sum[wave & 1][q * 16 + m][(4 * g + i) * 8 + half * 4]);
                        f32x4_t v = k * f32x4_t{acc[4 * half][q][i], acc[4 * half + 1][q][i],
                                                acc[4 * half + 2][q][i], acc[4 * half + 3][q][i]};
                        if (turn == 1)
                            v += *d;
                        *d = v;
                    }
            }
        __syncthreads();
    }
    const float factor = !is_a && a.l.scales ? a.l.scales[tile.a] : 1.0f;
    const int64_t size_a = (int64_t)a.R * a.K;
    float *part = nullptr;  // fp32 output: partials, or the caller's
    uint16_t *out16 = nullptr;
    const int64_t out0 = (int64_t)tile.a * a.R * C;
    if (chunks > 1)
        part = a.partials + (int64_t)(tile.slot + tile.index) * ((a.K + (int64_t)a.N) * a.R) +
               (is_a ? 0 : size_a);
    else if (a.fp32_out)
        part = static_cast<float *>(is_a ? a.dA : a.dB) + out0;
    else
        out16 = static_cast<uint16_t *>(is_a ? a.dA : a.dB) + out0;
    auto sum_of = [&](int r, int x) {
        const float v = s_sum[0][r][x] + s_sum[1][r][x];
        return rt * kRanks + r < rank ? factor * v : 0.0f;
    };
    auto put = [&](int64_t to, float v) {
        if (part)
            part[to] = v;
        else
            out16[to] = Elem<DT>::narrow(v);
    };
    // A thread takes pieces of 8 columns of dA's rows, of 4 ranks of dB's.  The
    // piece that reaches past column C was moved back: its own columns begin at
    // `back`, in LDS as everywhere.
    const int ranks_here = min(kRanks, a.R - rt * kRanks);
    if (is_a) {
        for (int i = threadIdx.x; i < kRanks * 16; i += 256) {
            const int r = i / 16, x = i % 16 * 8;
            const int c = ct * 128 + x;
            if (r >= ranks_here || c >= C)
                continue;
            const int64_t to = (int64_t)(rt * kRanks + r) * C + min(c, C - 8);
            const int back = max(c - (C - 8), 0);
            if (back == 0) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = sum_of(r, x + e);
                if (part) {
                    *reinterpret_cast<f32x4u_t *>(part + to) = f32x4_t{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4u_t *>(part + to + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
                } else {
                    typename Pack16<DT>::vec_t o;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = Elem<DT>::narrow(v[e]);
                    *reinterpret_cast<typename Pack16<DT>::vec_t *>(out16 + to) = o;
                }
            } else {
                for (int e = back; e < 8; ++e)
                    put(to + e, sum_of(r, x + e));
            }
        }
    } else {
        for (int i = threadIdx.x; i < kRanks / 4 * 128; i += 256) {
            const int r = i % (kRanks / 4) * 4, x = i / (kRanks / 4);
            const int c = ct * 128 + x;
            if (r >= ranks_here || c >= C)
                continue;
            const int back = max(ct * 128 + x / 8 * 8 - (C - 8), 0);
            const int64_t to = (int64_t)c * a.R + rt * kRanks + r;
            if (r + 4 <= ranks_here) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = sum_of(r + e, x + back);
                if (part) {
                    *reinterpret_cast<f32x4u_t *>(part + to) = f32x4_t{v[0], v[1], v[2], v[3]};
                } else {
                    typedef uint16_t half_t __attribute__((ext_vector_type(4), aligned(2)));
                    *reinterpret_cast<half_t *>(out16 + to) =
                        half_t{Elem<DT>::narrow(v[0]), Elem<DT>::narrow(v[1]),
                               Elem<DT>::narrow(v[2]), Elem<DT>::narrow(v[3])};
                }
            } else {
                for (int e = 0; r + e < ranks_here; ++e)
                    put(to + e, sum_of(r + e, x + back));
            }
        }
    }
}

// h summed over the splits (dh for the gradients, where no expand sums it).
__global__ __launch_bounds__(256) void sum_splits_kernel(const float *h, float *out, int64_t n,
                                                         int splits)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n)
        return;
    float v = h[i];
    for (int s = 1; s < splits; ++s)
        v += h[s * n + i];
    out[i] = v;
}

// Adds the partials of adapters with several chunks, in chunk order, 4
// elements a thread (one where K or N times R is no multiple of 4).
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
    const int step = (size_a | size) % 4 == 0 ? 4 : 1;
    for (int64_t i = ((int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x) * step; i < size;
         i += (int64_t)blocks * 256 * step) {
        const bool is_a = i < size_a;
        void *const out = is_a ? a.dA : a.dB;
        const int64_t to = is_a ? (int64_t)tile.a * size_a + i
                                : (int64_t)tile.a * a.R * a.N + (i - size_a);
        f32x4_t v = {};
        if (step == 4) {
            for (int c = 0; c < chunks; ++c)
                v += *reinterpret_cast<const f32x4u_t *>(part + c * size + i);
        } else {
            for (int c = 0; c < chunks; ++c)
                v[0] += part[c * size + i];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e >= step)
                break;
            if (a.fp32_out)
                static_cast<float *>(out)[to + e] = v[e];
            else
                static_cast<uint16_t *>(out)[to + e] = Elem<DT>::narrow(v[e]);
        }
    }
}

// ---------------------------------------------------------------- launches

template <int DT, bool TR, int RF, int RT>
hipError_t shrink_rt(const LoraParams &p, int64_t tiles, hipStream_t stream)
{
    const dim3 grid((unsigned)(tiles * p.splits)), block(kShrinkWaves * kWave);
    if (p.C % 32 || p.R % 4 || (TR && p.R % RF))
        hipLaunchKernelGGL((shrink_kernel<DT, TR, RF, RT, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((shrink_kernel<DT, TR, RF, RT, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int DT, bool TR, int RF> hipError_t shrink_rf(const LoraParams &p, hipStream_t stream)
{
    constexpr int kMany = shrink_blocks(RF * 16);
    const int rows = lora_shrink_rows(p.T, p.L, p.R);
    const int64_t tiles = (p.T + rows - 1) / rows + (p.T < p.L ? p.T : p.L);
    if (rows > 16)
        return shrink_rt<DT, TR, RF, kMany>(p, tiles, stream);
    return shrink_rt<DT, TR, RF, 1>(p, tiles, stream);
}

template <int DT, bool TR> hipError_t shrink_go(const LoraParams &p, hipStream_t stream)
{
    if (p.R <= 16)
        return shrink_rf<DT, TR, 1>(p, stream);
    if (p.R <= 32)
        return shrink_rf<DT, TR, 2>(p, stream);
    if (p.R <= 64)
        return shrink_rf<DT, TR, 4>(p, stream);
    if (p.R <= 128)
        return shrink_rf<DT, TR, 8>(p, stream);
    return shrink_rf<DT, TR, 16>(p, stream);
}

template <int DT, bool TR, int NS, bool SMALL, int RT>
hipError_t expand_rt(const LoraParams &p, hipStream_t stream)
{
    // As many passes a workgroup as leave one workgroup for each place on the
    // chip (expand_places a compute unit, by its registers): a workgroup takes 4 us before its first
    // pass, and a second, short round of workgroups would cost a whole one.
    const int64_t tiles = (p.T + RT * 16 - 1) / (RT * 16) + (p.T < p.L ? p.T : p.L);
    const int pass = 4 * 64;
    const int most = (p.C + pass - 1) / pass;
    const int64_t places = 256 * expand_places(TR, NS, RT);
    const int64_t passes = (most * tiles + places - 1) / places;
    int groups = (int)((most + passes - 1) / passes);
    const int group_cols = ((p.C + groups - 1) / groups + pass - 1) / pass * pass;
    groups = (p.C + group_cols - 1) / group_cols;
    const dim3 grid((unsigned)(tiles * groups)), block(256);
    if (p.C % 64 || p.R % 8)
        hipLaunchKernelGGL((expand_kernel<DT, TR, NS, SMALL, RT, true>), grid, block, 0, stream, p,
                           groups, group_cols);
    else
        hipLaunchKernelGGL((expand_kernel<DT, TR, NS, SMALL, RT, false>), grid, block, 0, stream, p,
                           groups, group_cols);
    return hipGetLastError();
}

template <int DT, bool TR, int NS, bool SMALL>
hipError_t expand_ns(const LoraParams &p, hipStream_t stream)
{
    return lora_many_rows(p.T, p.L) ? expand_rt<DT, TR, NS, SMALL, 4>(p, stream)
                                    : expand_rt<DT, TR, NS, SMALL, 1>(p, stream);
}

template <int DT, bool TR> hipError_t expand_go(const LoraParams &p, hipStream_t stream)
{
    if (p.R <= 16)
        return expand_ns<DT, TR, 1, true>(p, stream);
    if (p.R <= 32)
        return expand_ns<DT, TR, 1, false>(p, stream);
    if (p.R <= 64)
        return expand_ns<DT, TR, 2, false>(p, stream);
    if (p.R <= 128)
        return expand_ns<DT, TR, 4, false>(p, stream);
    return expand_ns<DT, TR, 8, false>(p, stream);
}

template <int DT> hipError_t grad_go(const GradParams &p, hipStream_t stream)
{
    const int64_t items = p.l.L + p.l.T / p.chunk;
    const int64_t rank_tiles = lora_rank_tiles(p.R);
    const dim3 grid((unsigned)(items * (p.col_tiles_a + p.col_tiles_b) * rank_tiles));
    if (p.R <= 16)
        hipLaunchKernelGGL((grad_kernel<DT, 1>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((grad_kernel<DT, 2>), grid, dim3(256), 0, stream, p);
    if (p.l.T <= p.chunk)
        return hipGetLastError();
    // Up to 1024 elements a workgroup and adapter, at most about 16 workgroups
    // a compute unit.
    const int64_t size = (int64_t)p.R * ((int64_t)p.K + p.N);
    int64_t blocks = (size + 1023) / 1024;
    const int64_t most = (4096 + p.l.L - 1) / p.l.L;
    blocks = blocks < most ? blocks : most;
    hipLaunchKernelGGL((grad_join_kernel<DT>), dim3((unsigned)(p.l.L * blocks)), dim3(256), 0,
                       stream, p, (int)blocks);
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

hipError_t lora_sum_launch(const float *h, float *out, int64_t n, int splits, hipStream_t stream)
{
    hipLaunchKernelGGL(sum_splits_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream,
                       h, out, n, splits);
    return hipGetLastError();
}

hipError_t lora_grad_launch(const GradParams &p, int dtype, hipStream_t stream)
{
    return dtype == kBf16 ? grad_go<kBf16>(p, stream) : grad_go<kFp16>(p, stream);
}

}  // namespace moegg
