// The gated feed-forward block's backward, gfx950 (moegg_gated_bwd): dH = dY_e W_e
// of the down projection (reduction over N) with the gated activation's backward
// as its epilogue.
#include "block_epilogue.h"

namespace moegg {

// Stages of the main loop.
constexpr int kBwdDepth = 64, kBwdStages = 2;

template <class C, bool PACKED, bool TAIL>
__global__ __launch_bounds__(C::NT) void gated_bwd_kernel(GatedBwdParams a)
{
    typedef Ring<C, kBwdDepth, kBwdStages> R;
    typedef RingLoader<C::BM, C::NT, kBwdDepth> LoadA;
    typedef RingTileLoader<C::BN, C::NT, kBwdDepth> LoadB;
    __shared__ __attribute__((aligned(16))) char smem[R::BYTES];
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(smem));
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[C::BM];
    __shared__ int s_scratch[2];

    const bool py = a.flags & MOEGG_PERMUTE_Y;
    const bool halves = a.flags & MOEGG_GATED_HALVES;
    const GateAct act(a.flags & MOEGG_GATED_GELU);
    const int nti = (a.I + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return (m + C::BM - 1) / C::BM * nti; });
    const int N = a.N;
    const int nsteps = (N + kBwdDepth - 1) / kBwdDepth;
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
        LoadA la;
        LoadB lb;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], a.ldy);
        lb.init(i0, a.I, a.ldw);
        ring_loop<C, kBwdDepth, kBwdStages, true, LoadA::RPT + LoadB::RPT>(
            lds, nsteps, acc,
            [&](int s, int n, uint32_t to) {
                if (n < LoadA::RPT)
                    la.issue(dyr, n, to, s * kBwdDepth, N);
                else
                    lb.issue(wr, n - LoadA::RPT, to + R::A, s * kBwdDepth, N);
            },
            rows);

        const int I = a.I;
        const int64_t Ip = packed_cols(I);
        for_constants<C::FM>([&](auto i) {
            const int64_t dst = s_dst[wm * C::TM + i * 32 + (lane & 31)];
            for_constants<C::FN>([&](auto j) {
                uint32_t d[16];
                row_cols(acc[i][j], d);
                const int blk = i0 + wn * C::TN + j * 32;
                const int col = blk + 16 * (lane >> 5);
                if (dst >= 0 && col < I) {
                    float g[16], u[16], h[16];
                    if constexpr (PACKED) {
                        const char *q = a.Aq + dst * 2 * Ip + col;
                        const uint8_t *s = a.As + (dst * 2 * Ip + blk) / kPackBlock;
                        unpack_cols(*reinterpret_cast<const uint4 *>(q), s[0], g);
                        unpack_cols(*reinterpret_cast<const uint4 *>(q + Ip), s[Ip / kPackBlock], u);
                    } else {
                        load_planes<TAIL>(a.A + dst * I * 4, col, I, halves, g, u);
                    }
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float dh = __uint_as_float(d[q]);
                        float v, slope;
                        act.slope(g[q], v, slope);
                        h[q] = v * u[q];
                        g[q] = dh * u[q] * slope;
                        u[q] = dh * v;
                    }
                    store_planes<TAIL>(a.dA + dst * I * 4, col, I, halves, g, u);
                    if (a.H)
                        store_cols<TAIL>(a.H + dst * I * 2, col, I, h);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        __syncthreads();
    }
}

using BwdBigCfg = Cfg<256, 256, 2, 4, true>;
using BwdSmallCfg = Cfg<32, 128, 1, 4, true>;

template <class C, bool PACKED, bool TAIL>
static void gated_bwd_cfg(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = row_tiles(p.S, p.E, C::BM) * ((p.I + C::BN - 1) / C::BN);
    static const int most = resident_workgroups(gated_bwd_kernel<C, PACKED, TAIL>, C::NT);
    const int64_t grid = std::max<int64_t>(1, std::min((int64_t)cus * most, tiles));
    hipLaunchKernelGGL((gated_bwd_kernel<C, PACKED, TAIL>), dim3((unsigned)grid), dim3(C::NT), 0,
                       stream, p);
}

template <bool PACKED, bool TAIL>
static void gated_bwd_rows(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    if (p.S / p.E < kBlockSmallRows)
        gated_bwd_cfg<BwdSmallCfg, PACKED, TAIL>(p, cus, stream);
    else
        gated_bwd_cfg<BwdBigCfg, PACKED, TAIL>(p, cus, stream);
}

hipError_t gated_bwd_launch(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    if (p.Aq) {
        if (p.I % 8)
            gated_bwd_rows<true, true>(p, cus, stream);
        else
            gated_bwd_rows<true, false>(p, cus, stream);
    } else {
        if (p.I % 8)
            gated_bwd_rows<false, true>(p, cus, stream);
        else
            gated_bwd_rows<false, false>(p, cus, stream);
    }
    return hipGetLastError();
}

}  // namespace moegg
