// The feed-forward block around the grouped products, gfx950:
//
//   block_fwd_kernel   Y = X W_e^T by 8-bit integers with a scale for each token
//                      and output channel, plain or gated; and the gated block in
//                      bf16, which can keep its pre-activations for the backward.
//   gated_bwd_kernel   dH = dY W_e of the down projection with the gated
//                      activation's backward as its epilogue.
//
// Both run the engine of gemm_engine.h with the MFMA's operands exchanged
// (Cfg::SWAP): a lane then holds 16 columns of one output row in each 32 x 32
// block, and one exchange with the lane 32 away makes them 16 neighbours
// (row_cols).  The epilogues work on those directly, without shared memory:
// scales, activation, block maxima and codes need no other lane but that one,
// and a row's 32 columns leave in whole 32- or 64-byte pieces.
#include "gemm_engine.h"

#include "block_params.h"
#include "pack.h"

namespace moegg {

// ---------------------------------------------------------------------------
// Epilogue pieces
// ---------------------------------------------------------------------------

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

// act(g) of the gated block: silu, or gelu by its tanh form, for which
// (1 + tanh z) / 2 = 1 / (1 + e^-2z).  v_exp_f32 and v_rcp_f32: an ulp each,
// far below the one rounding of the result to bf16.
__device__ __forceinline__ float gate_sigmoid(float g, bool gelu)
{
    const float z = gelu ? 1.5957691216057308f * g * (1.0f + 0.044715f * g * g) : g;
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
__device__ __forceinline__ float gate_act(float g, bool gelu)
{
    return g * gate_sigmoid(g, gelu);
}
// act(g) and act'(g): with s the sigmoid of z(g), act = g s and
// act' = s + g s (1 - s) z'.  Beyond |g| = 64 the sigmoid is 0 or 1 to the last
// bit, so that the slope is taken there, where no product overflows.
__device__ __forceinline__ void gate_act_slope(float g, bool gelu, float &a, float &slope)
{
    const float c = fminf(fmaxf(g, -64.0f), 64.0f);
    const float s = gate_sigmoid(c, gelu);
    const float dz = gelu ? 1.5957691216057308f * (1.0f + 3.0f * 0.044715f * c * c) : 1.0f;
    a = gate_act(g, gelu);
    slope = g != g ? g : s + c * s * (1.0f - s) * dz;
}

// Columns [col, col + 16) of a bf16 row of n elements.
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
        if (c + 8 <= n)
            *reinterpret_cast<u16x8_any_t *>(row + (int64_t)c * 2) = v;
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < n)
                    *reinterpret_cast<uint16_t *>(row + (int64_t)(c + i) * 2) = v[i];
    }
}

// The same columns of two planes of width n, as (first, second) neighbours
// (pairs) or as the halves of a row of 2 n.
__device__ __forceinline__ void store_planes(char *row, int col, int n, bool halves,
                                             const float (&f)[16], const float (&s)[16])
{
    if (halves) {
        store_cols(row, col, n, f);
        store_cols(row + (int64_t)n * 2, col, n, s);
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
    store_cols(row, 2 * col, 2 * n, a);
    store_cols(row, 2 * col + 16, 2 * n, b);
}

__device__ __forceinline__ void load_cols(const char *row, int col, int n, float (&f)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = col + 8 * h;
        u16x8_any_t v = {};
        if (c + 8 <= n)
            v = *reinterpret_cast<const u16x8_any_t *>(row + (int64_t)c * 2);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < n)
                    v[i] = *reinterpret_cast<const uint16_t *>(row + (int64_t)(c + i) * 2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[8 * h + i] = __builtin_bit_cast(float, (uint32_t)v[i] << 16);
    }
}

__device__ __forceinline__ void load_planes(const char *row, int col, int n, bool halves,
                                            float (&f)[16], float (&s)[16])
{
    if (halves) {
        load_cols(row, col, n, f);
        load_cols(row + (int64_t)n * 2, col, n, s);
        return;
    }
    float a[16], b[16];
    load_cols(row, 2 * col, 2 * n, a);
    load_cols(row, 2 * col + 16, 2 * n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = a[2 * i];
        s[i] = a[2 * i + 1];
        f[8 + i] = b[2 * i];
        s[8 + i] = b[2 * i + 1];
    }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// GATED: tile rows of W (columns of the output) are gate and up columns, whose
// accumulator blocks j and j + FN / 2 hold the same output columns (gated_row).
template <class C, bool GATED>
__device__ __forceinline__ int block_w_row(int n0, int r, int N, bool halves)
{
    int w = n0 + r;
    if constexpr (GATED) {
        w = n0 + gated_row<C>(r);
        if (halves) {  // pair (w / 2, w % 2) of an even n0
            const int o = w >> 1;
            w = o < N / 2 ? o + (w & 1) * (N / 2) : N;
        }
    }
    return w < N ? w : -1;
}

template <class C, bool GATED>
__global__ __launch_bounds__(C::NT) void block_fwd_kernel(BlockFwdParams a)
{
    __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
    char *const st0 = smem, *const st1 = smem + C::STAGE;
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[C::BM];
    __shared__ float s_scale[C::BM];
    __shared__ __attribute__((aligned(16))) float s_wscale[C::I8 ? C::BN : 4];
    __shared__ int s_scratch[2];

    const bool px = a.flags & MOEGG_PERMUTE_X, py = a.flags & MOEGG_PERMUTE_Y;
    const bool fm = a.flags & MOEGG_FUSE_MUL_POST;
    const bool gelu = a.flags & MOEGG_GATED_GELU, halves = a.flags & MOEGG_GATED_HALVES;
    const int ntn = (a.N + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return (m + C::BM - 1) / C::BM * ntn; });
    const int nsteps = (a.K + BK - 1) / BK;
    const int64_t x_rows = px ? a.S / a.topk : a.S;
    const u32x4_t xr = rsrc_words(a.X, x_rows * a.ldx);
    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int lane = threadIdx.x & (kWave - 1);

    for (int t = xcd_logical_block(blockIdx.x, gridDim.x); t < total; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[e + 1] - s_roff[e]);
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[e]);
        int mt, nt;
        band_raster<kBandM>(u, (mc + C::BM - 1) / C::BM, ntn, mt, nt);
        const int p0 = __builtin_amdgcn_readfirstlane(s_roff[e]) + mt * C::BM;
        const int rows = min(C::BM, mc - mt * C::BM);
        const int n0 = nt * C::BN;
        for (int i = threadIdx.x; i < C::BM; i += C::NT) {
            int src = -1, dst = -1;
            float scale = 1.0f;
            if (i < rows) {
                const int p = p0 + i;
                const int g = (px || py) ? checked_gather(a.gather, p, a.S, a.err) : p;
                if (g >= 0) {
                    src = px ? g / a.topk : p;
                    dst = py ? g : p;
                    if constexpr (C::I8)
                        scale = a.x_scales[src];
                    if (fm)
                        scale *= a.topk_w[g];
                }
            }
            s_src[i] = src;
            s_dst[i] = dst;
            s_scale[i] = scale;
        }
        if constexpr (C::I8)
            for (int r = threadIdx.x; r < C::BN; r += C::NT) {
                const int w = block_w_row<C, GATED>(n0, r, a.N, halves);
                s_wscale[r] = w < 0 ? 0.0f : a.w_scales[(int64_t)e * a.N + w];
            }
        __syncthreads();

        const u32x4_t wr = rsrc_words(a.W + (int64_t)e * a.N * a.ldw, (int64_t)a.N * a.ldw);
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        DmaLoader<C::BM, C::NT> la;
        DmaLoader<C::BN, C::NT> lb;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], a.ldx);
#pragma unroll
        for (int i = 0; i < lb.RPT; ++i)
            lb.set_row(i, block_w_row<C, GATED>(n0, lb.tile_row(i), a.N, halves), a.ldw);
        mainloop<C, true, false, false>(
            st0, st1, nsteps, acc,
            [&](int s, char *As, char *Bs) {
                la.load(xr, As, s * BK, a.K);
                lb.load(wr, Bs, s * BK, a.K);
            },
            rows);

        // This lane's 16 columns of row lane % 32 of each block.
        auto block = [&](int i, int j, float (&f)[16]) {
            uint32_t v[16];
            row_cols(acc[i][j], v);
            if constexpr (C::I8) {
                const float rs = s_scale[wm * C::TM + i * 32 + (lane & 31)];
                const float4 *ws = reinterpret_cast<const float4 *>(
                    s_wscale + wn * C::TN + j * 32 + 16 * (lane >> 5));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 w = ws[q];
                    f[4 * q] = (float)(int)v[4 * q] * rs * w.x;
                    f[4 * q + 1] = (float)(int)v[4 * q + 1] * rs * w.y;
                    f[4 * q + 2] = (float)(int)v[4 * q + 2] * rs * w.z;
                    f[4 * q + 3] = (float)(int)v[4 * q + 3] * rs * w.w;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    f[q] = __builtin_bit_cast(float, v[q]);
            }
        };
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int64_t dst = s_dst[wm * C::TM + i * 32 + (lane & 31)];
            if constexpr (!GATED) {
#pragma unroll
                for (int j = 0; j < C::FN; ++j) {
                    float f[16];
                    block(i, j, f);
                    const int col = n0 + wn * C::TN + j * 32 + 16 * (lane >> 5);
                    if (dst >= 0 && col < a.N)
                        store_cols(a.Y + dst * a.N * 2, col, a.N, f);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                constexpr int H = C::FN / 2;
                const int I = a.N / 2;
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    float g[16], v[16], h[16];
                    block(i, j, g);
                    block(i, j + H, v);
                    const int col = n0 / 2 + wn * (C::TN / 2) + j * 32 + 16 * (lane >> 5);
                    const int blk = n0 / 2 + wn * (C::TN / 2) + j * 32;
                    if constexpr (!C::I8) {
                        if (a.Aq) {
                            // Both lanes of a row take part; the block is outside when it starts at or past I.
                            const int64_t Ip = packed_cols(I);
                            uint4 gq, vq;
                            const uint8_t gs = pack_cols(g, gq), vs = pack_cols(v, vq);
                            if (dst >= 0 && blk < I) {
                                char *q = a.Aq + dst * 2 * Ip + col;
                                *reinterpret_cast<uint4 *>(q) = gq;
                                *reinterpret_cast<uint4 *>(q + Ip) = vq;
                                uint8_t *s = a.As + (dst * 2 * Ip + blk) / kPackBlock;
                                if (lane < 32)
                                    s[0] = gs;
                                else
                                    s[Ip / kPackBlock] = vs;
                            }
                        }
                        if (a.A && dst >= 0 && col < I)
                            store_planes(a.A + dst * a.N * 2, col, I, halves, g, v);
                    }
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        h[q] = gate_act(g[q], gelu) * v[q];
                    if (dst >= 0 && col < I)
                        store_cols(a.Y + dst * I * 2, col, I, h);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// dH = dY_e W_e (reduction over N) and the gated activation's backward
// ---------------------------------------------------------------------------

template <class C>
__global__ __launch_bounds__(C::NT) void gated_bwd_kernel(GatedBwdParams a)
{
    __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
    char *const st0 = smem, *const st1 = smem + C::STAGE;
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[C::BM];
    __shared__ int s_scratch[2];

    const bool py = a.flags & MOEGG_PERMUTE_Y;
    const bool gelu = a.flags & MOEGG_GATED_GELU, halves = a.flags & MOEGG_GATED_HALVES;
    const int nti = (a.I + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return (m + C::BM - 1) / C::BM * nti; });
    const int N = a.N;
    const int nsteps = (N + BK - 1) / BK;
    const u32x4_t dyr = rsrc_words(a.dY, a.S * a.ldy);
    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int lane = threadIdx.x & (kWave - 1);

    for (int t = xcd_logical_block(blockIdx.x, gridDim.x); t < total; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[e + 1] - s_roff[e]);
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[e]);
        int mt, it;
        band_raster<kBandMdX>(u, (mc + C::BM - 1) / C::BM, nti, mt, it);
        const int p0 = __builtin_amdgcn_readfirstlane(s_roff[e]) + mt * C::BM;
        const int rows = min(C::BM, mc - mt * C::BM);
        const int i0 = it * C::BN;
        for (int i = threadIdx.x; i < C::BM; i += C::NT) {
            int src = -1, dst = -1;
            if (i < rows) {
                const int p = p0 + i;
                const int g = py ? checked_gather(a.gather, p, a.S, a.err) : p;
                if (g >= 0) {
                    src = g;
                    dst = p;
                }
            }
            s_src[i] = src;
            s_dst[i] = dst;
        }
        __syncthreads();

        const u32x4_t wr = rsrc_words(a.W + (int64_t)e * N * a.ldw, (int64_t)N * a.ldw);
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        DmaLoader<C::BM, C::NT> la;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], a.ldy);
        TileDmaLoader<C::BN, C::NT> lb;
        auto wraw = [](int n) -> int { return n; };
        auto wfin = [=](int n, int) -> int { return n < N ? n : -1; };
        lb.fetch(0, wraw);
        mainloop<C, true, false, true>(
            st0, st1, nsteps, acc,
            [&](int s, char *As, char *Bs) {
                lb.prepare(i0, a.I, a.ldw, wfin);
                __builtin_amdgcn_sched_barrier(0);
                la.load(dyr, As, s * BK, N);
                lb.issue(wr, Bs);
                lb.fetch((s + 1) * BK, wraw);
            },
            rows);

        const int I = a.I;
        const int64_t Ip = packed_cols(I);
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int64_t dst = s_dst[wm * C::TM + i * 32 + (lane & 31)];
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                uint32_t d[16];
                row_cols(acc[i][j], d);
                const int blk = i0 + wn * C::TN + j * 32;
                const int col = blk + 16 * (lane >> 5);
                if (dst >= 0 && col < I) {
                    float g[16], v[16], dg[16], h[16];
                    if (a.Aq) {
                        const char *q = a.Aq + dst * 2 * Ip + col;
                        const uint8_t *s = a.As + (dst * 2 * Ip + blk) / kPackBlock;
                        unpack_cols(*reinterpret_cast<const uint4 *>(q), s[0], g);
                        unpack_cols(*reinterpret_cast<const uint4 *>(q + Ip), s[Ip / kPackBlock], v);
                    } else {
                        load_planes(a.A + dst * I * 4, col, I, halves, g, v);
                    }
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float dh = __builtin_bit_cast(float, d[q]);
                        float act, slope;
                        gate_act_slope(g[q], gelu, act, slope);
                        dg[q] = dh * v[q] * slope;
                        h[q] = act * v[q];
                        v[q] = dh * act;
                    }
                    store_planes(a.dA + dst * I * 4, col, I, halves, dg, v);
                    if (a.H)
                        store_cols(a.H + dst * I * 2, col, I, h);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------

// Tile shapes: many rows per expert, and few (the weights are then streamed
// once per 32-row tile).
using I8BigCfg = Cfg<256, 256, 2, 4, true, true>;
using I8SmallCfg = Cfg<32, 128, 1, 4, true, true>;
using I8SmallGatedCfg = Cfg<32, 256, 1, 4, true, true>;
using BlockBigCfg = Cfg<256, 256, 2, 4, true>;
using BlockSmallCfg = Cfg<32, 256, 1, 4, true>;
using BlockBwdSmallCfg = Cfg<32, 128, 1, 4, true>;

template __global__ void block_fwd_kernel<I8BigCfg, false>(BlockFwdParams);
template __global__ void block_fwd_kernel<I8SmallCfg, false>(BlockFwdParams);
template __global__ void block_fwd_kernel<I8BigCfg, true>(BlockFwdParams);
template __global__ void block_fwd_kernel<I8SmallGatedCfg, true>(BlockFwdParams);
template __global__ void block_fwd_kernel<BlockBigCfg, true>(BlockFwdParams);
template __global__ void block_fwd_kernel<BlockSmallCfg, true>(BlockFwdParams);
template __global__ void gated_bwd_kernel<BlockBigCfg>(GatedBwdParams);
template __global__ void gated_bwd_kernel<BlockBwdSmallCfg>(GatedBwdParams);

// Average rows per expert below which the small tiles are used, as for the
// bf16 products.
constexpr int64_t kBlockSmallRows = 96;

template <class Kern>
static int block_grid(Kern kernel, int threads, int64_t tiles, int cus)
{
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != hipSuccess || n < 1)
        n = 1;
    const int64_t g = std::min((int64_t)cus * n, tiles);
    return (int)std::max<int64_t>(g, 1);
}

static int64_t row_tiles(int64_t rows, int E, int block)
{
    return rows <= E ? rows : (rows - E + 1 + block - 1) / block + E - 1;
}

template <class C, bool GATED>
static void block_fwd_cfg(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = row_tiles(p.S, p.E, C::BM) * ((p.N + C::BN - 1) / C::BN);
    hipLaunchKernelGGL((block_fwd_kernel<C, GATED>),
                       dim3(block_grid(block_fwd_kernel<C, GATED>, C::NT, tiles, cus)), dim3(C::NT),
                       0, stream, p);
}

hipError_t i8_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const bool small = p.S / p.E < kBlockSmallRows;
    if (p.flags & (MOEGG_GATED_SILU | MOEGG_GATED_GELU)) {
        if (small)
            block_fwd_cfg<I8SmallGatedCfg, true>(p, cus, stream);
        else
            block_fwd_cfg<I8BigCfg, true>(p, cus, stream);
    } else {
        if (small)
            block_fwd_cfg<I8SmallCfg, false>(p, cus, stream);
        else
            block_fwd_cfg<I8BigCfg, false>(p, cus, stream);
    }
    return hipGetLastError();
}

hipError_t gated_fwd_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.S / p.E < kBlockSmallRows)
        block_fwd_cfg<BlockSmallCfg, true>(p, cus, stream);
    else
        block_fwd_cfg<BlockBigCfg, true>(p, cus, stream);
    return hipGetLastError();
}

template <class C>
static void gated_bwd_cfg(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = row_tiles(p.S, p.E, C::BM) * ((p.I + C::BN - 1) / C::BN);
    hipLaunchKernelGGL(gated_bwd_kernel<C>,
                       dim3(block_grid(gated_bwd_kernel<C>, C::NT, tiles, cus)), dim3(C::NT), 0,
                       stream, p);
}

hipError_t gated_bwd_launch(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    if (p.S / p.E < kBlockSmallRows)
        gated_bwd_cfg<BlockBwdSmallCfg>(p, cus, stream);
    else
        gated_bwd_cfg<BlockBigCfg>(p, cus, stream);
    return hipGetLastError();
}

}  // namespace moegg
