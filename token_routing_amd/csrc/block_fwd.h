// Y = grouped X W_e^T for the feed-forward block: by 8-bit integers with a scale
// for each token and output channel, plain or gated, and the gated block in
// bf16 with what its backward pass needs.
//
// Weights and rows come as 16-byte pieces of the reduction for both types, so that
// the int8 product is the bf16 loop with another MFMA and half the bytes.  Measured:
//   int8, 8192 rows of 4096 into 28672, gated    0.96 ms, 2.0 POP/s (the library's
//                                                int8 product at 8192^3: 2.15)
//   int8, 65536 rows of 768 into 2048            0.20 ms, 520 MB: loop 0.1, stores 0.1
//   int8, 512 rows over 128 experts, 2048 into 1536, gated   74 us, 5.4 TB/s of W
//   bf16, 65536 rows of 2048 into 2 x 768, A kept            0.50 ms, 0.82 PFLOP/s
//   bf16, 8192 rows of 4096 into 2 x 14336, packed           1.87 ms, 1.03 PFLOP/s
#pragma once

#include "block_epilogue.h"

namespace moegg {

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

// What a gated call keeps of its pre-activations.
constexpr int kKeepNone = 0, kKeepBf16 = 1, kKeepPacked = 2;

template <class C, int ACT, int KEEP, bool TAIL>
__global__ __launch_bounds__(C::NT) void block_fwd_kernel(BlockFwdParams a)
{
    typedef RingLoader<C::BM, C::NT, C::DEPTH> LoadA;
    typedef RingLoader<C::BN, C::NT, C::DEPTH> LoadB;
    constexpr int CPS = LoadA::RPT + LoadB::RPT;
    constexpr bool GATED = ACT != kPlain;
    typedef GateAct<ACT == kGelu> Act;
    // Tables of two tiles: this one's and the next one's.
    constexpr int WS = C::I8 ? C::BN : 4;
    __shared__ __attribute__((aligned(16))) char smem[C::BYTES];
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[2][C::BM];
    __shared__ float s_scale[2][C::BM];
    __shared__ __attribute__((aligned(16))) float s_wscale[2][WS];
    __shared__ int s_scratch[2];
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(smem));

    const bool px = a.flags & MOEGG_PERMUTE_X, py = a.flags & MOEGG_PERMUTE_Y;
    const bool fm = a.flags & MOEGG_FUSE_MUL_POST;
    const bool halves = a.flags & MOEGG_GATED_HALVES;
    const int ntn = (a.N + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return tiles_of<C::BM>(m) * ntn; });
    const int K = a.K, nsteps = (K + C::DEPTH - 1) / C::DEPTH;
    const int64_t x_rows = px ? a.S / a.topk : a.S;
    const u32x4_t xr = rsrc_words(a.X, x_rows * a.ldx);
    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int lane = threadIdx.x & (kWave - 1);

    // Tile t: its expert, first sorted position, real rows and first column.
    struct Tile {
        int e, p0, rows, n0;
    };
    auto locate = [&](int t) -> Tile {
        Tile x;
        x.e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[x.e + 1] - s_roff[x.e]);
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[x.e]);
        int mt, nt;
        band_raster<kBandM>(u, tiles_of<C::BM>(mc), ntn, mt, nt);
        x.p0 = __builtin_amdgcn_readfirstlane(s_roff[x.e]) + mt * C::BM;
        x.rows = min(C::BM, mc - mt * C::BM);
        x.n0 = nt * C::BN;
        return x;
    };
    // Gather entry of tile row threadIdx.x of tile t (-2: none), read before the
    // epilogue of the tile in front of it.
    static_assert(C::BM <= C::NT && WS <= 2 * C::NT, "tables filled in one pass");
    auto fetch = [&](int t) -> int {
        if (t >= total)
            return -2;
        const Tile x = locate(t);
        const int i = threadIdx.x;
        if (i >= C::BM || i >= x.rows)
            return -2;
        return (px || py) ? a.gather[x.p0 + i] : x.p0 + i;
    };
    // The loaders of a tile, and its scales, on the way in registers.
    LoadA la;
    LoadB lb;
    u32x4_t wr;
    float row_scale = 1.0f, w_scale[2] = {0.0f, 0.0f};
    auto copy = [&](int s, int n, uint32_t to) {
        if (n < LoadA::RPT)
            la.issue(xr, n, to, s * C::DEPTH, K);
        else
            lb.issue(wr, n - LoadA::RPT, to + C::A, s * C::DEPTH, K);
    };
    auto start = [&](const Tile &x, int g, int buf) {
        if (threadIdx.x < C::BM) {
            int src = -1, dst = -1;
            row_scale = 1.0f;
            if (g != -2) {
                if ((px || py) && (g < 0 || g >= a.S)) {
                    raise_error(a.err, kErrGather);
                } else {
                    const int p = x.p0 + threadIdx.x;
                    src = px ? g / a.topk : p;
                    dst = py ? g : p;
                    if constexpr (C::I8)
                        row_scale = a.x_scales[src];
                    if (fm)
                        row_scale *= a.topk_w[g];
                }
            }
            s_src[threadIdx.x] = src;
            s_dst[buf][threadIdx.x] = dst;
        }
        if constexpr (C::I8)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = threadIdx.x + h * C::NT;
                const int w = r < WS ? block_w_row<C, GATED>(x.n0, r, a.N, halves) : -1;
                w_scale[h] = w < 0 ? 0.0f : a.w_scales[(int64_t)x.e * a.N + w];
            }
        __syncthreads();
        wr = rsrc_words(a.W + (int64_t)x.e * a.N * a.ldw, (int64_t)a.N * a.ldw);
#pragma unroll
        for (int i = 0; i < LoadA::RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], a.ldx);
#pragma unroll
        for (int i = 0; i < LoadB::RPT; ++i)
            lb.set_row(i, block_w_row<C, GATED>(x.n0, lb.tile_row(i), a.N, halves), a.ldw);
        ring_start<C, CPS>(lds, nsteps, copy);
    };

    int t = xcd_logical_block(blockIdx.x, gridDim.x), buf = 0;
    if (t >= total)
        return;
    Tile x = locate(t);
    start(x, fetch(t), 0);
    int g = fetch(t + gridDim.x);
    for (;;) {
        if constexpr (C::I8) {
            if (threadIdx.x < C::BM)
                s_scale[buf][threadIdx.x] = row_scale;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (threadIdx.x + h * C::NT < WS)
                    s_wscale[buf][threadIdx.x + h * C::NT] = w_scale[h];
        }
        const int tn = t + gridDim.x;
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        ring_loop<C, false, CPS>(lds, nsteps, acc, copy, x.rows);
        const int n0 = x.n0;
        if (tn < total) {
            x = locate(tn);
            start(x, g, buf ^ 1);
            g = fetch(tn + gridDim.x);
        }

        // This lane's 16 columns of row lane % 32 of a block.
        auto block = [&](auto i, auto j, float (&f)[16]) {
            uint32_t v[16];
            row_cols(acc[i][j], v);
            if constexpr (C::I8) {
                const float rs = s_scale[buf][wm * C::TM + i * 32 + (lane & 31)];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 w = *reinterpret_cast<const float4 *>(
                        s_wscale[buf] + wn * C::TN + j * 32 + lane_col(q / 2) + q % 2 * 4);
                    f[4 * q] = (float)(int)v[4 * q] * rs * w.x;
                    f[4 * q + 1] = (float)(int)v[4 * q + 1] * rs * w.y;
                    f[4 * q + 2] = (float)(int)v[4 * q + 2] * rs * w.z;
                    f[4 * q + 3] = (float)(int)v[4 * q + 3] * rs * w.w;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    f[q] = __uint_as_float(v[q]);
            }
        };
        constexpr int H = GATED ? C::FN / 2 : C::FN;
        const int cols = GATED ? a.N / 2 : a.N;
        const int c0 = (GATED ? n0 / 2 + wn * (C::TN / 2) : n0 + wn * C::TN);
        for_constants<C::FM>([&](auto i) {
            const int64_t dst = s_dst[buf][wm * C::TM + i * 32 + (lane & 31)];
            uint32_t gbytes = 0, ubytes = 0;
            for_constants<H>([&](auto j) {
                const int blk = c0 + j * 32;
                float f[16];
                block(i, j, f);
                if constexpr (GATED) {
                    float u[16];
                    block(i, std::integral_constant<int, decltype(j)::value + H>{}, u);
                    if constexpr (KEEP == kKeepPacked) {
                        const int64_t Ip = packed_cols(cols);
                        uint32_t gq[4], uq[4];
                        gbytes |= pack_cols(f, gq) << (8 * j);
                        ubytes |= pack_cols(u, uq) << (8 * j);
                        exchange_codes(gq);
                        exchange_codes(uq);
                        // Whole blocks: columns past the last one are zeros.
                        if (dst >= 0 && blk < cols) {
                            char *q = a.Aq + dst * 2 * Ip + blk + 16 * (lane >> 5);
                            *reinterpret_cast<uint4 *>(q) = uint4{gq[0], gq[1], gq[2], gq[3]};
                            *reinterpret_cast<uint4 *>(q + Ip) = uint4{uq[0], uq[1], uq[2], uq[3]};
                        }
                    }
                    if constexpr (KEEP == kKeepBf16)
                        if (dst >= 0)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (blk + lane_col(h) < cols)
                                    store8_planes<TAIL>(a.A + dst * a.N * 2, blk + lane_col(h), cols,
                                                        halves, f + 8 * h, u + 8 * h);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        f[q] = Act::act(f[q]) * u[q];
                }
                if (dst >= 0)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (blk + lane_col(h) < cols)
                            store8<TAIL>(a.Y + dst * cols * 2, blk + lane_col(h), cols, f + 8 * h);
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (KEEP == kKeepPacked) {
                // The row's bytes of these blocks: the gate's from one lane, the other's
                // from the other.
                const int64_t nb = packed_cols(cols) / kPackBlock;
                const uint32_t w = lane < 32 ? gbytes : ubytes;
                uint8_t *s = a.As + dst * 2 * nb + (lane < 32 ? 0 : nb) + c0 / kPackBlock;
                if (dst >= 0)
#pragma unroll
                    for (int j = 0; j < H; ++j)
                        if (c0 + j * 32 < cols)
                            s[j] = (uint8_t)(w >> (8 * j));
            }
        });
        if (tn >= total)
            return;
        t = tn;
        buf ^= 1;
    }
}

template <class C, int ACT, int KEEP, bool TAIL>
void block_fwd_cfg(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = row_tiles(p.S, p.E, C::BM) * ((p.N + C::BN - 1) / C::BN);
    static const int most = resident_workgroups(block_fwd_kernel<C, ACT, KEEP, TAIL>, C::NT);
    const int64_t grid = std::max<int64_t>(1, std::min((int64_t)cus * most, tiles));
    hipLaunchKernelGGL((block_fwd_kernel<C, ACT, KEEP, TAIL>), dim3((unsigned)grid), dim3(C::NT),
                       0, stream, p);
}

}  // namespace moegg
