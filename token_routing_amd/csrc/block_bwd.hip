// The gated feed-forward block's backward, gfx950 (moegg_gated_bwd): dH = dY_e W_e
// of the down projection (reduction over N) with the gated activation's backward
// as its epilogue.
//
// dH stays in registers in fp32, so that it costs neither its rounding nor its 2 S I
// bytes each way.  W's rows are the reduction: its tiles go to LDS as they are and are
// read transposed (ds_read_b64_tr_b16).  65536 rows of 2048 into 768 with 8-bit kept
// values: 367 us (0.56 PFLOP/s, 2.9 TB/s), where the product bounds it at 133 us and
// its bytes at 214; from bf16 406 us (233 of bytes).  8192 rows of 4096 into 14336 1.2 ms
// (0.80 PFLOP/s), from bf16 1.26.  3003 odd rows, 1003 into 517: 34 us, from bf16 37, of
// which copying the operands in front takes 11.  Main loop and epilogue (kept values in, dA
// and H out) follow each other on a compute unit.
#include "block_epilogue.h"

namespace moegg {

// 16 gate and linear values of a row as they were kept, and their values.
template <bool PACKED, bool TAIL>
struct Kept;

template <bool TAIL>
struct Kept<true, TAIL> {
    uint4 g, u;
    uint32_t gs, us;
    __device__ __forceinline__ void load(const char *q, const uint8_t *s, int64_t Ip)
    {
        g = *reinterpret_cast<const uint4 *>(q);
        u = *reinterpret_cast<const uint4 *>(q + Ip);
        gs = s[0];
        us = s[Ip / kPackBlock];
    }
    // To the columns of row_cols; all lanes take part.
    __device__ __forceinline__ void arrange()
    {
        uint32_t w[4] = {g.x, g.y, g.z, g.w}, v[4] = {u.x, u.y, u.z, u.w};
        exchange_codes(w);
        exchange_codes(v);
        g = uint4{w[0], w[1], w[2], w[3]};
        u = uint4{v[0], v[1], v[2], v[3]};
    }
    // Columns 8 h .. + 7 of the 16.
    __device__ __forceinline__ void values(int h, bool, float (&f)[8], float (&v)[8]) const
    {
        unpack_cols(h ? g.z : g.x, h ? g.w : g.y, gs, f);
        unpack_cols(h ? u.z : u.x, h ? u.w : u.y, us, v);
    }
};

template <bool TAIL>
struct Kept<false, TAIL> {
    u16x8_any_t w[4];  // of columns 8 h .. + 7: two of them
    __device__ __forceinline__ void load(const char *row, int blk, int n, bool halves)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = blk + lane_col(h);
            if (c >= n)
                continue;
            if (halves) {
                w[2 * h] = load8<TAIL>(row, c, n);
                w[2 * h + 1] = load8<TAIL>(row + (int64_t)n * 2, c, n);
            } else {
                w[2 * h] = load8<TAIL>(row, 2 * c, 2 * n);
                w[2 * h + 1] = load8<TAIL>(row, 2 * c + 8, 2 * n);
            }
        }
    }
    __device__ __forceinline__ void arrange() {}
    __device__ __forceinline__ void values(int h, bool halves, float (&f)[8], float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t hf = w[2 * h][i], hv = w[2 * h + 1][i];
            const uint32_t pf = w[2 * h + i / 4][i % 4 * 2], pv = w[2 * h + i / 4][i % 4 * 2 + 1];
            f[i] = __uint_as_float((halves ? hf : pf) << 16);
            v[i] = __uint_as_float((halves ? hv : pv) << 16);
        }
    }
};

template <class C, bool GELU, bool PACKED, bool TAIL>
__global__ __launch_bounds__(C::NT) void gated_bwd_kernel(GatedBwdParams a)
{
    typedef RingLoader<C::BM, C::NT, C::DEPTH> LoadA;
    typedef RingTileLoader<C::BN, C::NT, C::DEPTH> LoadB;
    constexpr int CPS = LoadA::RPT + LoadB::RPT;
    __shared__ __attribute__((aligned(16))) char smem[C::BYTES];
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[2][C::BM];  // this tile's and the next one's
    __shared__ int s_scratch[2];
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_u32(smem));

    const bool py = a.flags & MOEGG_PERMUTE_Y;
    const bool halves = a.flags & MOEGG_GATED_HALVES;
    const int nti = (a.I + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return tiles_of<C::BM>(m) * nti; });
    const int N = a.N, nsteps = (N + C::DEPTH - 1) / C::DEPTH;
    const u32x4_t dyr = rsrc_words(a.dY, a.S * a.ldy);
    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int lane = threadIdx.x & (kWave - 1);

    // Tile t: its expert, first sorted position, real rows and first column.
    struct Tile {
        int e, p0, rows, i0;
    };
    auto locate = [&](int t) -> Tile {
        Tile x;
        x.e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[x.e + 1] - s_roff[x.e]);
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[x.e]);
        int mt, it;
        band_raster<kBandMdX>(u, tiles_of<C::BM>(mc), nti, mt, it);
        x.p0 = __builtin_amdgcn_readfirstlane(s_roff[x.e]) + mt * C::BM;
        x.rows = min(C::BM, mc - mt * C::BM);
        x.i0 = it * C::BN;
        return x;
    };
    // Gather entry of tile row threadIdx.x of tile t (-2: none), read before the
    // epilogue of the tile in front of it.
    static_assert(C::BM <= C::NT, "tables filled in one pass");
    auto fetch = [&](int t) -> int {
        if (t >= total)
            return -2;
        const Tile x = locate(t);
        const int i = threadIdx.x;
        if (i >= C::BM || i >= x.rows)
            return -2;
        return py ? a.gather[x.p0 + i] : x.p0 + i;
    };
    LoadA la;
    LoadB lb;
    u32x4_t wr;
    auto copy = [&](int s, int n, uint32_t to) {
        if (n < LoadA::RPT)
            la.issue(dyr, n, to, s * C::DEPTH, N);
        else
            lb.issue(wr, n - LoadA::RPT, to + C::A, s * C::DEPTH, N);
    };
    auto start = [&](const Tile &x, int g, int buf) {
        if (threadIdx.x < C::BM) {
            int src = -1, dst = -1;
            if (g != -2) {
                if (py && (g < 0 || g >= a.S)) {
                    raise_error(a.err, kErrGather);
                } else {
                    src = g;
                    dst = x.p0 + threadIdx.x;
                }
            }
            s_src[threadIdx.x] = src;
            s_dst[buf][threadIdx.x] = dst;
        }
        __syncthreads();
        wr = rsrc_words(a.W + (int64_t)x.e * N * a.ldw, (int64_t)N * a.ldw);
#pragma unroll
        for (int i = 0; i < LoadA::RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], a.ldy);
        lb.init(x.i0, a.I, a.ldw);
        ring_start<C, CPS>(lds, nsteps, copy);
    };

    int t = xcd_logical_block(blockIdx.x, gridDim.x), buf = 0;
    if (t >= total)
        return;
    Tile x = locate(t);
    start(x, fetch(t), 0);
    int g = fetch(t + gridDim.x);
    for (;;) {
        const int tn = t + gridDim.x;
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        ring_loop<C, true, CPS>(lds, nsteps, acc, copy, x.rows);
        const int i0 = x.i0;
        if (tn < total) {
            x = locate(tn);
            start(x, g, buf ^ 1);
            g = fetch(tn + gridDim.x);
        }

        const int I = a.I;
        const int64_t Ip = packed_cols(I);
        // What was kept of block (i, j)'s columns, its loads issued before the stores of the
        // block in front of them.  Loads and stores stand under conditions of the lane, which
        // the compiler cannot count: it waits for everything in flight, from packed values at
        // every second block, from bf16 at each load.
        Kept<PACKED, TAIL> kept[2];
        auto load = [&](auto b) {
            constexpr int i = decltype(b)::value / C::FN, j = decltype(b)::value % C::FN;
            const int64_t dst = s_dst[buf][wm * C::TM + i * 32 + (lane & 31)];
            const int blk = i0 + wn * C::TN + j * 32;
            if (dst < 0 || blk >= I)
                return;
            if constexpr (PACKED)
                kept[decltype(b)::value & 1].load(a.Aq + dst * 2 * Ip + blk + 16 * (lane >> 5),
                                                  a.As + (dst * 2 * Ip + blk) / kPackBlock, Ip);
            else
                kept[decltype(b)::value & 1].load(a.A + dst * I * 4, blk, I, halves);
        };
        constexpr int NB = C::FM * C::FN;
        load(std::integral_constant<int, 0>{});
        for_constants<NB>([&](auto b) {
            constexpr int i = decltype(b)::value / C::FN, j = decltype(b)::value % C::FN;
            if constexpr (b + 1 < NB)
                load(std::integral_constant<int, b + 1>{});
            const int64_t dst = s_dst[buf][wm * C::TM + i * 32 + (lane & 31)];
            uint32_t d[16];
            row_cols(acc[i][j], d);
            kept[b & 1].arrange();
            for_constants<2>([&](auto h) {
                const int c = i0 + wn * C::TN + j * 32 + lane_col(h);
                if (dst >= 0 && c < I) {
                    float g[8], u[8], o[8];
                    kept[b & 1].values(h, halves, g, u);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float dh = __uint_as_float(d[8 * h + q]);
                        float v, slope;
                        GateAct<GELU>::slope(g[q], v, slope);
                        o[q] = v * u[q];
                        g[q] = dh * u[q] * slope;
                        u[q] = dh * v;
                    }
                    store8_planes<TAIL>(a.dA + dst * I * 4, c, I, halves, g, u);
                    if (a.H)
                        store8<TAIL>(a.H + dst * I * 2, c, I, o);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        if (tn >= total)
            return;
        t = tn;
        buf ^= 1;
    }
}

using BwdBigCfg = RingCfg<256, 256, 2, 4, false, 64, 2>;
using BwdMidCfg = RingCfg<128, 128, 2, 2, false, 64, 2>;
using BwdDeepCfg = RingCfg<128, 128, 2, 2, false, 64, 4>;
using BwdSmallCfg = RingCfg<32, 128, 1, 4, false, 64, 4>;

template <class C, bool GELU, bool PACKED, bool TAIL>
static void gated_bwd_cfg(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = row_tiles(p.S, p.E, C::BM) * ((p.I + C::BN - 1) / C::BN);
    static const int most = resident_workgroups(gated_bwd_kernel<C, GELU, PACKED, TAIL>, C::NT);
    const int64_t grid = std::max<int64_t>(1, std::min((int64_t)cus * most, tiles));
    hipLaunchKernelGGL((gated_bwd_kernel<C, GELU, PACKED, TAIL>), dim3((unsigned)grid), dim3(C::NT), 0,
                       stream, p);
}

template <bool GELU, bool PACKED, bool TAIL>
static void gated_bwd_rows(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    constexpr bool TWO = PACKED && !TAIL;
    const Shape shape = bwd_shape(p.S, p.E, p.I, BwdSmallCfg::BN, 0.9, TWO, cus);
    if (shape == kSmallTiles)
        return gated_bwd_cfg<BwdSmallCfg, GELU, PACKED, TAIL>(p, cus, stream);
    if (shape == kBigTiles)
        return gated_bwd_cfg<BwdBigCfg, GELU, PACKED, TAIL>(p, cus, stream);
    if constexpr (TWO)
        if (shape == kMidTiles)
            return gated_bwd_cfg<BwdMidCfg, GELU, PACKED, TAIL>(p, cus, stream);
    gated_bwd_cfg<BwdDeepCfg, GELU, PACKED, TAIL>(p, cus, stream);
}

template <bool GELU, bool PACKED>
static void gated_bwd_tail(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    if (p.I % 8)
        gated_bwd_rows<GELU, PACKED, true>(p, cus, stream);
    else
        gated_bwd_rows<GELU, PACKED, false>(p, cus, stream);
}

template <bool GELU>
static void gated_bwd_kept(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    if (p.Aq)
        gated_bwd_tail<GELU, true>(p, cus, stream);
    else
        gated_bwd_tail<GELU, false>(p, cus, stream);
}

hipError_t gated_bwd_launch(const GatedBwdParams &p, int cus, hipStream_t stream)
{
    if (p.flags & MOEGG_GATED_GELU)
        gated_bwd_kept<true>(p, cus, stream);
    else
        gated_bwd_kept<false>(p, cus, stream);
    return hipGetLastError();
}

}  // namespace moegg
