// Y = grouped X W_e^T for the feed-forward block: by 8-bit integers with a scale
// for each token and output channel, plain or gated, and the gated block in
// bf16 with what its backward pass needs.
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

// Stages of the main loop.
constexpr int kFwdDepth = 64, kFwdStages = 2;

template <class C, bool GATED, int KEEP, bool TAIL>
__global__ __launch_bounds__(C::NT) void block_fwd_kernel(BlockFwdParams a)
{
    typedef Ring<C, kFwdDepth, kFwdStages> R;
    typedef RingLoader<C::BM, C::NT, kFwdDepth> LoadA;
    typedef RingLoader<C::BN, C::NT, kFwdDepth> LoadB;
    __shared__ __attribute__((aligned(16))) char smem[R::BYTES];
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(smem));
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[C::BM];
    __shared__ float s_scale[C::BM];
    __shared__ __attribute__((aligned(16))) float s_wscale[C::I8 ? C::BN : 4];
    __shared__ int s_scratch[2];

    const bool px = a.flags & MOEGG_PERMUTE_X, py = a.flags & MOEGG_PERMUTE_Y;
    const bool fm = a.flags & MOEGG_FUSE_MUL_POST;
    const bool halves = a.flags & MOEGG_GATED_HALVES;
    const GateAct act(a.flags & MOEGG_GATED_GELU);
    const int ntn = (a.N + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return (m + C::BM - 1) / C::BM * ntn; });
    const int nsteps = (a.K + kFwdDepth - 1) / kFwdDepth;
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
        LoadA la;
        LoadB lb;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], a.ldx);
#pragma unroll
        for (int i = 0; i < lb.RPT; ++i)
            lb.set_row(i, block_w_row<C, GATED>(n0, lb.tile_row(i), a.N, halves), a.ldw);
        const int K = a.K;
        ring_loop<C, kFwdDepth, kFwdStages, false, LoadA::RPT + LoadB::RPT>(
            lds, nsteps, acc,
            [&](int s, int n, uint32_t to) {
                if (n < LoadA::RPT)
                    la.issue(xr, n, to, s * kFwdDepth, K);
                else
                    lb.issue(wr, n - LoadA::RPT, to + R::A, s * kFwdDepth, K);
            },
            rows);

        // This lane's 16 columns of row lane % 32 of a block.
        auto block = [&](auto i, auto j, float (&f)[16]) {
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
                    f[q] = __uint_as_float(v[q]);
            }
        };
        constexpr int H = GATED ? C::FN / 2 : C::FN;
        const int cols = GATED ? a.N / 2 : a.N;
        const int c0 = (GATED ? n0 / 2 + wn * (C::TN / 2) : n0 + wn * C::TN);
        for_constants<C::FM>([&](auto i) {
            const int64_t dst = s_dst[wm * C::TM + i * 32 + (lane & 31)];
            for_constants<H>([&](auto j) {
                const int blk = c0 + j * 32, col = blk + 16 * (lane >> 5);
                float f[16];
                block(i, j, f);
                if constexpr (GATED) {
                    float u[16];
                    block(i, std::integral_constant<int, decltype(j)::value + H>{}, u);
                    if constexpr (KEEP == kKeepPacked) {
                        const int64_t Ip = packed_cols(cols);
                        uint4 gq, uq;
                        const uint32_t gs = pack_cols(f, gq), us = pack_cols(u, uq);
                        // Whole blocks: the lane past the last column writes zeros.
                        if (dst >= 0 && blk < cols) {
                            char *q = a.Aq + dst * 2 * Ip + col;
                            *reinterpret_cast<uint4 *>(q) = gq;
                            *reinterpret_cast<uint4 *>(q + Ip) = uq;
                            uint8_t *s = a.As + (dst * 2 * Ip + blk) / kPackBlock +
                                         (lane < 32 ? 0 : Ip / kPackBlock);
                            *s = (uint8_t)(lane < 32 ? gs : us);
                        }
                    }
                    if constexpr (KEEP == kKeepBf16)
                        if (dst >= 0 && col < cols)
                            store_planes<TAIL>(a.A + dst * a.N * 2, col, cols, halves, f, u);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        f[q] = act(f[q]) * u[q];
                }
                if (dst >= 0 && col < cols)
                    store_cols<TAIL>(a.Y + dst * cols * 2, col, cols, f);
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        __syncthreads();
    }
}

template <class C, bool GATED, int KEEP, bool TAIL>
void block_fwd_cfg(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = row_tiles(p.S, p.E, C::BM) * ((p.N + C::BN - 1) / C::BN);
    static const int most = resident_workgroups(block_fwd_kernel<C, GATED, KEEP, TAIL>, C::NT);
    const int64_t grid = std::max<int64_t>(1, std::min((int64_t)cus * most, tiles));
    hipLaunchKernelGGL((block_fwd_kernel<C, GATED, KEEP, TAIL>), dim3((unsigned)grid), dim3(C::NT),
                       0, stream, p);
}

}  // namespace moegg
