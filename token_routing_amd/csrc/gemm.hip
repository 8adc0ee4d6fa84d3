// Persistent grouped-GEMM kernels for gfx950: forward (with permute_x,
// permute_y, fuse_mul_post and the gated activation), dX, dW (ragged
// reduction per expert, optionally split for hot experts) and explicit GEMM
// groups.
//
// The operations are those of grouped_gemm_forward / grouped_gemm_dX /
// grouped_gemm_dW (unsloth grouped_gemm/interface.py), whose per-expert
// meaning is the loop of matmul_ogs_torch (triton_kernels/matmul_ogs.py), and
// of asym_dual_gmm_separated (wall_x/fusions/backend.py) for the groups.
//
// The engine is in gemm_engine.h.
#include <type_traits>

#include "gemm_engine.h"

namespace moegg {

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// GATED: W rows come in (gate, linear) pairs and Y gets N/2 columns of the
// gated activation (epilogue_gated).
template <class C, bool GATED>
__global__ __launch_bounds__(C::NT) void fwd_kernel(FwdParams a)
{
    __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
    char *const st0 = smem, *const st1 = smem + C::STAGE;
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[C::BM];
    __shared__ float s_scale[C::BM];
    __shared__ int s_scratch[2];

    const bool px = a.flags & MOEGG_PERMUTE_X, py = a.flags & MOEGG_PERMUTE_Y;
    const bool fm = a.flags & MOEGG_FUSE_MUL_POST;
    const int ntn = (a.N + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return tiles_of<C::BM>(m) * ntn; });
    const int nsteps = (a.K + BK - 1) / BK;
    const int64_t row_bytes = (int64_t)a.K * 2;
    const int64_t x_rows = px ? a.S / a.topk : a.S;
    const u32x4_t xr = rsrc_words(a.X, x_rows * row_bytes);

    // Tile t: expert, first sorted position, real rows, first column.
    auto tile = [&](int t, int &e, int &p0, int &rows, int &n0) {
        e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[e + 1] - s_roff[e]);
        const int mtiles = tiles_of<C::BM>(mc);
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[e]);
        int mt, nt;
        band_raster<kBandM>(u, mtiles, ntn, mt, nt);
        p0 = __builtin_amdgcn_readfirstlane(s_roff[e]) + mt * C::BM;
        rows = min(C::BM, mc - mt * C::BM);
        n0 = nt * C::BN;
    };
    // Gather entry of tile row threadIdx.x (one row per thread; -2: none).
    // The next tile's entry is loaded before this tile's mainloop, so its
    // latency is hidden; only the gate factor, which depends on it, is read
    // when the tile starts.
    static_assert(C::BM <= C::NT, "one tile row per thread");
    auto fetch = [&](int p0, int rows) -> int {
        const int i = threadIdx.x;
        if (i >= C::BM || i >= rows)
            return -2;
        return (px || py) ? a.gather[p0 + i] : p0 + i;
    };

    int t = xcd_logical_block(blockIdx.x, gridDim.x);
    int e = 0, p0 = 0, rows = 0, n0 = 0, g = -2;
    if (t < total) {
        tile(t, e, p0, rows, n0);
        g = fetch(p0, rows);
    }
    for (; t < total; t += gridDim.x) {
        if (threadIdx.x < C::BM) {
            const int i = threadIdx.x;
            int src = -1, dst = -1;
            float scale = 1.0f;
            if (g != -2) {
                const int64_t p = p0 + i;
                if ((px || py) && (g < 0 || g >= a.S)) {
                    raise_error(a.err, kErrGather);
                } else {
                    src = px ? g / a.topk : (int)p;
                    dst = py ? g : (int)p;
                    if (fm)
                        scale = a.topk_w[g];
                }
            }
            s_src[i] = src;
            s_dst[i] = dst;
            s_scale[i] = scale;
        }
        __syncthreads();
        // The next tile's gather entries, in flight during this mainloop.
        const int tn = t + gridDim.x;
        int e_n = 0, p0_n = 0, rows_n = 0, n0_n = 0, g_n = -2;
        if (tn < total) {
            tile(tn, e_n, p0_n, rows_n, n0_n);
            g_n = fetch(p0_n, rows_n);
        }

        const u32x4_t wr =
            rsrc_words(a.W + (int64_t)e * a.N * row_bytes, (int64_t)a.N * row_bytes);
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        DmaLoader<C::BM, C::NT> la;
        DmaLoader<C::BN, C::NT> lb;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], row_bytes);
#pragma unroll
        for (int i = 0; i < lb.RPT; ++i) {
            const int r = lb.tile_row(i);
            int wrow = n0 + r;
            if constexpr (GATED)
                wrow = n0 + gated_row<C>(r);
            lb.set_row(i, wrow < a.N ? wrow : -1, row_bytes);
        }
        mainloop<C, true, false, false>(
            st0, st1, nsteps, acc,
            [&](int s, char *As, char *Bs) {
                la.load(xr, As, s * BK, a.K);
                lb.load(wr, Bs, s * BK, a.K);
            },
            rows);
        if constexpr (GATED)
            epilogue_gated<C>(st0, acc, s_dst, a.Y, a.N / 2, n0 / 2, a.N / 2);
        else
            epilogue_bf16<C, true>(st0, st1, acc, s_dst, s_scale, a.Y, a.N, n0, a.N);
        e = e_n;
        p0 = p0_n;
        rows = rows_n;
        n0 = n0_n;
        g = g_n;
    }
}

// ---------------------------------------------------------------------------
// dX = dY_e W_e  (reduction over N)
// ---------------------------------------------------------------------------

template <class C>
__global__ __launch_bounds__(C::NT) void dx_kernel(DxParams a)
{
    __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
    char *const st0 = smem, *const st1 = smem + C::STAGE;
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_src[C::BM];
    __shared__ int s_dst[C::BM];
    __shared__ int s_scratch[2];

    const bool px = a.flags & MOEGG_PERMUTE_X, py = a.flags & MOEGG_PERMUTE_Y;
    const int ntk = (a.K + C::BN - 1) / C::BN;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return (m + C::BM - 1) / C::BM * ntk; });
    const int nsteps = (a.N + BK - 1) / BK;
    const int64_t dy_row = (int64_t)a.N * 2, w_row = (int64_t)a.K * 2;
    const u32x4_t dyr = rsrc_words(a.dY, a.S * dy_row);
    const TailPlan tp = tail_plan(total, gridDim.x, a.ws != nullptr);
    int32_t *const hdr = reinterpret_cast<int32_t *>(a.ws);
    if (a.ws && blockIdx.x == 0 && threadIdx.x == 0) {
        hdr[0] = tp.R;
        hdr[1] = tp.P;
    }

    for (int w = xcd_logical_block(blockIdx.x, gridDim.x); w < tp.items; w += gridDim.x) {
        int t, part;
        tail_item(tp, w, t, part);
        const int e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[e + 1] - s_roff[e]);
        const int p0base = __builtin_amdgcn_readfirstlane(s_roff[e]);
        const int mtiles = (mc + C::BM - 1) / C::BM;
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[e]);
        int mt, kt;
        band_raster<kBandMdX>(u, mtiles, ntk, mt, kt);
        const int p0 = p0base + mt * C::BM;
        const int rows = min(C::BM, mc - mt * C::BM);
        const int k0 = kt * C::BN;
        // A tail part reduces its share of the N range into a partial whose
        // row i is tile row i (the finishing launch maps rows to dX).
        const bool tail = part >= 0;
        const int r = t - tp.full;
        if (tail && part == 0 && threadIdx.x == 0) {
            hdr[2 + 4 * r] = p0;
            hdr[3 + 4 * r] = rows;
            hdr[4 + 4 * r] = k0;
            hdr[5 + 4 * r] = e;
        }

        for (int i = threadIdx.x; i < C::BM; i += C::NT) {
            int src = -1, dst = -1;
            if (i < rows) {
                const int64_t p = p0 + i;
                const int g = (px || py) ? checked_gather(a.gather, p, a.S, a.err) : (int)p;
                if (g >= 0) {
                    src = py ? g : (int)p;
                    dst = px ? g : (int)p;
                }
            }
            s_src[i] = src;
            s_dst[i] = tail ? i : dst;
        }
        __syncthreads();
        float *const partial =
            tail ? reinterpret_cast<float *>(a.ws + tail_header_bytes()) +
                       (int64_t)(r * tp.P + part) * C::BM * C::BN
                 : nullptr;

        const u32x4_t wr =
            rsrc_words(a.W + (int64_t)e * a.N * w_row, (int64_t)a.N * w_row);
        f32x16_t acc[C::FM][C::FN];
        if constexpr (UseQuad<C>::value) {
            // Wave w copies dY rows [64 w, 64 w + 64) (A, reduction-contiguous)
            // and W rows 8 w .. 8 w + 7 of each slot (B, row-major).
            using Q = Quad<C>;
            const int first = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * 64;
            SlotCopier<Q::NCA> ca;
            SlotTileCopier<C::BN, Q::NCB> cb;
            ca.init(smem, first);
#pragma unroll
            for (int j = 0; j < Q::NCA; ++j)
                ca.set_row(j, s_src[ca.row(first, j)], dy_row);
            cb.init(smem + Q::A, 0, k0, a.K, w_row);
            const int N = a.N;
            const int U = (N + SK - 1) / SK;
            const int u0 = tail ? part * U / tp.P : 0, u1 = tail ? (part + 1) * U / tp.P : U;
            zero_acc<C>(acc);
            mainloop_quad<C, false, true>(
                smem, u1 - u0, acc,
                plain_copy([&](int q, int buf, int n) {
                    const int qq = q + u0;
                    if (n < Q::NCA)
                        ca.template issue_one<Q::SLOT>(dyr, n, buf, qq * SK, N);
                    else
                        cb.template issue_one<Q::SLOT>(wr, n - Q::NCA, buf, qq, N);
                }),
                rows);
            if (tail) {
                epilogue_f32<C>(acc, s_dst, partial, C::BN, 0, C::BN);
                __syncthreads();
            } else {
                epilogue_bf16<C>(st0, st1, acc, s_dst, nullptr, a.dX, a.K, k0, a.K);
            }
            continue;
        }
        DmaLoader<C::BM, C::NT> la;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i)
            la.set_row(i, s_src[la.tile_row(i)], dy_row);
        const int N = a.N;
        const int u0 = tail ? part * nsteps / tp.P : 0;
        const int u1 = tail ? (part + 1) * nsteps / tp.P : nsteps;
        zero_acc<C>(acc);
        TileDmaLoader<C::BN, C::NT> lb;
        auto wraw = [](int n) -> int { return n; };
        auto wfin = [=](int n, int) -> int { return n < N ? n : -1; };
        lb.fetch(u0 * BK, wraw);
        mainloop<C, true, false, true>(
            st0, st1, u1 - u0, acc,
            [&](int s, char *As, char *Bs) {
                lb.prepare(k0, a.K, w_row, wfin);
                __builtin_amdgcn_sched_barrier(0);
                la.load(dyr, As, (s + u0) * BK, a.N);
                lb.issue(wr, Bs);
                lb.fetch((s + u0 + 1) * BK, wraw);
            },
            rows);
        if (tail) {
            epilogue_f32<C>(acc, s_dst, partial, C::BN, 0, C::BN);
            __syncthreads();
        } else {
            epilogue_bf16<C>(st0, st1, acc, s_dst, nullptr, a.dX, a.K, k0, a.K);
        }
    }
}

// ---------------------------------------------------------------------------
// dW_e = dY_e^T X_e  (reduction over the expert's own rows)
// ---------------------------------------------------------------------------

constexpr int kGroupK = 8;

// The copies of a 64-row stage take longer to land than the MFMAs of the
// previous stage run: with the MFMAs removed, the two-stage loop still takes
// 1.5 us per stage on the Mixtral shape, against 0.95 us per stage with the
// copies removed.  dW therefore splits the same 128 KiB of LDS into four
// 32-row slots and issues each slot's copies three slots ahead.  Gather
// entries are staged in LDS for a segment of up to kDwGather rows at a time,
// so that the only vector-memory operations in the loop are the copies and
// each wait can count them.  Measured: fine-grained dW 0.404 -> 0.368 ms,
// decode-shaped dW 0.113 -> 0.105 ms; the Mixtral shape is unchanged (its
// copies are bound by their rate, not by how far ahead they are issued).
constexpr int kDwSlot = 32;      // reduction rows per slot
constexpr int kDwSlots = 4;
constexpr int kDwGather = 1024;  // gather entries staged per segment

// MFMAs of one 32-row slot (both operands reduction rows in LDS).
template <class C>
__device__ __forceinline__ void dw_slot_mma(const char *As, const char *Bs,
                                            f32x16_t (&acc)[C::FM][C::FN], int wm, int wn)
{
    bf16x8_t a0[C::FM], b0[C::FN], a1[C::FM], b1[C::FN];
    read_step<C, true, true>(As, Bs, 0, wm, wn, a0, b0);
    read_step<C, true, true>(As, Bs, 1, wm, wn, a1, b1);
    mma_step<C>(a0, b0, acc);
    mma_step<C>(a1, b1, acc);
}


// PX / PY: the forward's permute flags, as template parameters so that the
// per-stage row-index code has no flag branches.
template <class C, bool PX, bool PY>
__global__ __launch_bounds__(C::NT) void dw_kernel(DwParams a)
{
    __shared__ __attribute__((aligned(16))) char smem[2 * C::STAGE];
    char *const st0 = smem, *const st1 = smem + C::STAGE;
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_order[kMaxExperts];
    __shared__ int s_crows[kMaxExperts];       // rows per chunk, by sorted position
    __shared__ int s_istart[kMaxExperts + 1];  // first work item, by sorted position
    __shared__ int s_poff[kMaxExperts + 1];    // first partial (split experts), by position
    __shared__ int s_dst[C::BM];
    __shared__ int s_scratch[4];

    const bool f32out = a.flags & MOEGG_DW_FP32_OUT;
    const int ntn = (a.N + C::BM - 1) / C::BM, ntk = (a.K + C::BN - 1) / C::BN;
    const int per_expert = ntn * ntk;
    build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                        [&](int) { return 0; });
    // Chunks: an expert longer than split_rows is cut into c chunks of cr
    // rows (a multiple of BK, the last one shorter); otherwise one chunk of
    // all its rows.  Work items (chunk x output tile) are ordered by chunk
    // length, longest first, so the long reductions start early.
    auto chunking = [&](int m, int &c, int &cr) {
        c = 1;
        cr = m;
        if (a.split_rows > 0 && m > a.split_rows) {
            c = (m + a.split_rows - 1) / a.split_rows;
            cr = ((m + c - 1) / c + BK - 1) / BK * BK;
            c = (m + cr - 1) / cr;
        }
    };
    int *const s_cnt = s_tstart;  // chunks by sorted position (s_tstart is free here)
    for (int e = threadIdx.x; e < a.E; e += C::NT) {
        int c, cr;
        chunking(s_roff[e + 1] - s_roff[e], c, cr);
        int rank = 0;
        for (int f = 0; f < a.E; ++f) {
            int cf, crf;
            chunking(s_roff[f + 1] - s_roff[f], cf, crf);
            rank += (crf > cr) || (crf == cr && f < e);
        }
        s_order[rank] = e;
        s_crows[rank] = cr;
        s_cnt[rank] = c;
        s_istart[rank] = c * per_expert;
        s_poff[rank] = c > 1 ? c : 0;
    }
    wave0_exclusive_scan(s_istart, a.E, &s_scratch[2]);
    wave0_exclusive_scan(s_poff, a.E, &s_scratch[3]);
    const int total = s_scratch[2];
    float *const partials =
        a.ws ? reinterpret_cast<float *>(a.ws + dw_header_bytes(a.E)) : nullptr;
    if (blockIdx.x == 0 && a.split_rows > 0 && a.ws) {
        // The plan for dw_reduce: split experts in sorted order.
        int32_t *hdr = reinterpret_cast<int32_t *>(a.ws);
        if (threadIdx.x < kWave) {
            int base = 0;
            for (int p0 = 0; p0 < a.E; p0 += kWave) {
                const int pos = p0 + threadIdx.x;
                const int cnt = pos < a.E ? s_cnt[pos] : 0;
                const bool split = cnt > 1;
                const uint64_t mask = __ballot(split);
                const int j = base + __popcll(mask & ((1ull << threadIdx.x) - 1));
                if (split) {
                    hdr[1 + 3 * j] = s_order[pos];
                    hdr[2 + 3 * j] = cnt;
                    hdr[3 + 3 * j] = s_poff[pos];
                }
                base += __popcll(mask);
            }
            if (threadIdx.x == 0)
                hdr[0] = base;
        }
    }
    const int64_t dy_row = (int64_t)a.N * 2, x_row = (int64_t)a.K * 2;
    const int64_t x_rows = PX ? a.S / a.topk : a.S;
    const u32x4_t dyr = rsrc_words(a.dY, a.S * dy_row);
    const u32x4_t xr = rsrc_words(a.X, x_rows * x_row);

    for (int t = xcd_logical_block(blockIdx.x, gridDim.x); t < total; t += gridDim.x) {
        const int pos = __builtin_amdgcn_readfirstlane(upper_index(s_istart, a.E, t));
        const int e = __builtin_amdgcn_readfirstlane(s_order[pos]);
        const int item = t - __builtin_amdgcn_readfirstlane(s_istart[pos]);
        const int chunk = item / per_expert;
        const int cr = __builtin_amdgcn_readfirstlane(s_crows[pos]);
        const int m_e = __builtin_amdgcn_readfirstlane(s_roff[e + 1] - s_roff[e]);
        const bool split = cr < m_e;  // chunked expert: fp32 partial into the workspace
        // Grouped raster inside the expert: runs of up to kGroupK K-panels per
        // N column, so consecutive tiles (one XCD's concurrent set) share
        // few dY (N) and X (K) panels in that XCD's L2.
        const int u = item % per_expert;
        const int span = kGroupK * ntn;
        const int first_kt = (u / span) * kGroupK;
        const int gk = min(ntk - first_kt, kGroupK);
        const int kt = first_kt + (u % span) % gk, nt = (u % span) / gk;
        const int n0 = nt * C::BM, k0 = kt * C::BN;
        const int start = __builtin_amdgcn_readfirstlane(s_roff[e]) + chunk * cr;
        const int mc = max(0, min(cr, m_e - chunk * cr));

        if (m_e == 0) {
            // An expert without rows: its tile of dW is zeros, stored as 16-byte
            // row segments straight from registers (no copies, MFMAs or LDS
            // staging; every thread of the workgroup takes this branch).
            const int esz = f32out ? 4 : 2;
            const int cpr = min(C::BN, a.K - k0) * esz / 16;  // K is a multiple of 8
            const int nrows = min(C::BM, a.N - n0);
            char *const base = a.dW + (((int64_t)e * a.N + n0) * a.K + k0) * esz;
            const u32x4_nt_t z = {0u, 0u, 0u, 0u};
            for (int idx = threadIdx.x; idx < nrows * cpr; idx += C::NT) {
                const int r = idx / cpr, c = idx % cpr;
                __builtin_nontemporal_store(
                    z, reinterpret_cast<u32x4_nt_t *>(base + (int64_t)r * a.K * esz + c * 16));
            }
            continue;
        }

        __syncthreads();
        for (int i = threadIdx.x; i < C::BM; i += C::NT)
            s_dst[i] = (n0 + i < a.N) ? (split ? 0 : e * a.N) + n0 + i : -1;
        __syncthreads();

        const int64_t S = a.S;
        const int32_t *gather = a.gather;
        int32_t *err = a.err;
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        {
            static_assert(kDwSlots * 2 * C::BM * kDwSlot * 2 <= 2 * C::STAGE &&
                              C::BM == C::BN && kMaxExperts + 1 >= kDwGather,
                          "four slots in the two stages; gather entries in s_tstart");
            constexpr int SLOT_A = C::BM * kDwSlot * 2, SLOT = 2 * SLOT_A;
            int *const s_g = s_tstart;  // free once the plan is built
            const FastDiv tdiv = a.topk_div;
            const uint32_t Su = (uint32_t)S;
            const int wave = threadIdx.x / kWave;
            const int wm = wave / C::WN, wn = wave % C::WN;
            bool bad = false;
            TileDmaLoader<C::BM, C::NT, kDwSlot> la;
            TileDmaLoader<C::BN, C::NT, kDwSlot> lb;
            constexpr int NC = TileDmaLoader<C::BM, C::NT, kDwSlot>::RPT +
                               TileDmaLoader<C::BN, C::NT, kDwSlot>::RPT;  // copies per wave per slot
            for (int seg0 = 0; seg0 < mc; seg0 += kDwGather) {
                const int segn = min(kDwGather, mc - seg0);
                const int ns = (segn + kDwSlot - 1) / kDwSlot;
                if constexpr (PX || PY) {
                    for (int i = threadIdx.x; i < segn; i += C::NT)
                        s_g[i] = gather[start + seg0 + i];
                    __syncthreads();
                } else {
                    wait_vmem();  // earlier stores: the waits below count copies only
                }
                // HBM rows of segment row r (-1: zeros).  A gather entry
                // outside [0, S) gives zeros and is reported once per tile.
                auto dyrow = [&](int r) -> int {
                    const bool in = r < segn;
                    if constexpr (PY) {
                        const int g = s_g[min(r, segn - 1)];
                        const bool ok = (uint32_t)g < Su;
                        bad |= in && !ok;
                        return in && ok ? g : -1;
                    }
                    return in ? start + seg0 + r : -1;
                };
                auto xrow = [&](int r) -> int {
                    const bool in = r < segn;
                    if constexpr (PX) {
                        const int g = s_g[min(r, segn - 1)];
                        const bool ok = (uint32_t)g < Su;
                        bad |= in && !ok;
                        return in && ok ? fast_div((uint32_t)g, tdiv) : -1;
                    }
                    return in ? start + seg0 + r : -1;
                };
                auto issue = [&](int q) {
                    char *sl = smem + (q % kDwSlots) * SLOT;
                    la.prepare_rows(n0, a.N, dy_row, [&](int row) { return dyrow(q * kDwSlot + row); });
                    lb.prepare_rows(k0, a.K, x_row, [&](int row) { return xrow(q * kDwSlot + row); });
                    __builtin_amdgcn_sched_barrier(0);
                    la.issue(dyr, sl);
                    lb.issue(xr, sl + SLOT_A);
                };
                for (int q = 0; q < min(ns, kDwSlots - 1); ++q)
                    issue(q);
                for (int q = 0; q < ns; ++q) {
                    // Slot q's copies are complete once at most the copies of
                    // the (up to two) slots issued after it are in flight.
                    const int after = min(kDwSlots - 2, ns - 1 - q);
                    if (after >= 2)
                        wait_vmcnt<2 * NC>();
                    else if (after == 1)
                        wait_vmcnt<NC>();
                    else
                        wait_vmcnt<0>();
                    wait_lds();
                    wg_barrier();
                    // Every wave is past slot q - 1, whose buffer slot q + 3 reuses.
                    if (q + kDwSlots - 1 < ns)
                        issue(q + kDwSlots - 1);
                    const char *sl = smem + (q % kDwSlots) * SLOT;
                    dw_slot_mma<C>(sl, sl + SLOT_A, acc, wm, wn);
                }
                __syncthreads();  // slots and s_g free for the next segment or the epilogue
            }
            if (bad)
                raise_error(err, kErrGather);
        }
        if (split) {
            const int poff = __builtin_amdgcn_readfirstlane(s_poff[pos]);
            epilogue_f32<C>(acc, s_dst, partials + (int64_t)(poff + chunk) * a.N * a.K, a.K, k0,
                            a.K);
        } else if (f32out) {
            epilogue_f32<C>(acc, s_dst, reinterpret_cast<float *>(a.dW), a.K, k0, a.K);
        } else {
            epilogue_bf16<C, false, true>(st0, st1, acc, s_dst, nullptr, a.dW, a.K, k0, a.K);
        }
    }
}

// Sums the chunk partials of the split experts in chunk order (fp32) into
// dW (bf16 or fp32), 16 bytes per lane and two positions per iteration (so
// that 2 c loads are in flight before the first add).  The plan comes from
// the workspace header written by dw_kernel's workgroup 0 earlier on the
// stream.
__device__ __forceinline__ void dw_reduce_store(const DwParams &a, int64_t o, const float4 &v)
{
    if (a.flags & MOEGG_DW_FP32_OUT) {
        reinterpret_cast<float4 *>(a.dW)[o] = v;
    } else {
        uint2 b;
        b.x = pack_bf16x2(v.x, v.y);
        b.y = pack_bf16x2(v.z, v.w);
        reinterpret_cast<uint2 *>(a.dW)[o] = b;
    }
}

__global__ __launch_bounds__(256) void dw_reduce_kernel(DwParams a)
{
    const int32_t *hdr = reinterpret_cast<const int32_t *>(a.ws);
    const float4 *partials = reinterpret_cast<const float4 *>(a.ws + dw_header_bytes(a.E));
    const int nsplit = hdr[0];
    const int64_t nk4 = (int64_t)a.N * a.K / 4;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int j = 0; j < nsplit; ++j) {
        const int e = hdr[1 + 3 * j], c = hdr[2 + 3 * j], p0 = hdr[3 + 3 * j];
        const float4 *src = partials + (int64_t)p0 * nk4;
        for (int64_t w = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; w < nk4; w += 2 * stride) {
            const bool two = w + stride < nk4;
            float4 s0 = src[w];
            float4 s1 = two ? src[w + stride] : float4{};
            for (int q = 1; q < c; ++q) {
                const float4 v0 = src[q * nk4 + w];
                const float4 v1 = two ? src[q * nk4 + w + stride] : float4{};
                s0.x += v0.x; s0.y += v0.y; s0.z += v0.z; s0.w += v0.w;
                s1.x += v1.x; s1.y += v1.y; s1.z += v1.z; s1.w += v1.w;
            }
            dw_reduce_store(a, (int64_t)e * nk4 + w, s0);
            if (two)
                dw_reduce_store(a, (int64_t)e * nk4 + w + stride, s1);
        }
    }
}

// ---------------------------------------------------------------------------
// Explicit groups: y_g = x_g @ w_g
// ---------------------------------------------------------------------------

// The groups are few short products (the dual-expert layer: one tile per CU,
// 16 stages over K = 1024): a tile's copies of one stage cannot hide their
// own latency behind one stage of MFMAs, so the groups run a four-stage ring.
constexpr int kGroupStages = 4;

template <class C, bool TRANS_B>
__global__ __launch_bounds__(C::NT) void groups_kernel(GroupsParams a)
{
    constexpr int NST = kGroupStages;
    __shared__ __attribute__((aligned(16))) char smem[NST * C::STAGE];
    char *const st0 = smem, *const st1 = smem + C::STAGE;
    __shared__ int s_tstart[MOEGG_MAX_GROUPS + 1];
    __shared__ int s_dst[C::BM];

    if (threadIdx.x == 0) {
        int run = 0;
        for (int i = 0; i < a.num; ++i) {
            s_tstart[i] = run;
            run += ((a.g[i].m + C::BM - 1) / C::BM) * ((a.g[i].n + C::BN - 1) / C::BN);
        }
        s_tstart[a.num] = run;
    }
    __syncthreads();
    const int total = s_tstart[a.num];

    for (int t = xcd_logical_block(blockIdx.x, gridDim.x); t < total; t += gridDim.x) {
        const int gi = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.num, t));
        const moegg_group &g = a.g[gi];
        const int mtiles = (g.m + C::BM - 1) / C::BM;
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[gi]);
        const int mt = u % mtiles, nt = u / mtiles;
        const int m0 = mt * C::BM, n0 = nt * C::BN;

        __syncthreads();
        for (int i = threadIdx.x; i < C::BM; i += C::NT)
            s_dst[i] = (m0 + i < g.m) ? m0 + i : -1;
        __syncthreads();

        const int64_t x_row = (int64_t)g.ldx * 2, w_row = (int64_t)g.ldw * 2;
        const u32x4_t xr = rsrc_words(g.x, (int64_t)g.m * x_row);
        const u32x4_t wr = rsrc_words(g.w, (int64_t)(TRANS_B ? g.n : g.k) * w_row);
        DmaLoader<C::BM, C::NT> la;
#pragma unroll
        for (int i = 0; i < la.RPT; ++i) {
            const int r = la.tile_row(i);
            la.set_row(i, m0 + r < g.m ? m0 + r : -1, x_row);
        }
        f32x16_t acc[C::FM][C::FN];
        zero_acc<C>(acc);
        const int nsteps = (g.k + BK - 1) / BK;
        const int kk = g.k;
        if constexpr (TRANS_B) {
            DmaLoader<C::BN, C::NT> lb;
#pragma unroll
            for (int i = 0; i < lb.RPT; ++i) {
                const int r = lb.tile_row(i);
                lb.set_row(i, n0 + r < g.n ? n0 + r : -1, w_row);
            }
            mainloop_ring<C, NST, false, false, decltype(la)::RPT + decltype(lb)::RPT>(
                smem, nsteps, acc,
                [&](int s, char *As, char *Bs) {
                    la.load(xr, As, s * BK, kk);
                    lb.load(wr, Bs, s * BK, kk);
                },
                min(C::BM, g.m - m0));
        } else {
            TileDmaLoader<C::BN, C::NT> lb;
            const int n = g.n;
            mainloop_ring<C, NST, false, true, decltype(la)::RPT + decltype(lb)::RPT>(
                smem, nsteps, acc,
                [&](int s, char *As, char *Bs) {
                    lb.prepare_rows(n0, n, w_row, [&](int row) {
                        const int red = s * BK + row;
                        return red < kk ? red : -1;
                    });
                    __builtin_amdgcn_sched_barrier(0);
                    la.load(xr, As, s * BK, kk);
                    lb.issue(wr, Bs);
                },
                min(C::BM, g.m - m0));
        }
        epilogue_bf16<C>(st0, st1, acc, s_dst, nullptr, static_cast<char *>(g.y), g.ldy, n0, g.n);
    }
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------

// Tile shapes: <BM, BN, waves along M, waves along N>.
using BigCfg = Cfg<256, 256, 2, 4>;     // many rows per expert
using DxCfg = Cfg<256, 256, 2, 4>;
using DxQuadCfg = Cfg<256, 256, 2, 2>;  // long reductions: four-wave engine
using DwCfg = Cfg<256, 256, 2, 4>;
using SmallCfg = Cfg<32, 128, 1, 4>;    // few rows per expert: stream the weights
using DxSmallCfg = Cfg<32, 128, 1, 4>;     // the same for dX
using SmallGatedCfg = Cfg<32, 256, 1, 4>;  // the same with two blocks per wave to pair
// Small explicit groups: tiles of 64 x 128 so that the dual-expert layer's
// 256 tiles cover every CU (128 x 128 tiles: 15.4 us against 11.9 us there;
// each tile's copies, about 0.4 MB over K = 1024, bound a CU's time).
using GroupCfg = Cfg<64, 128, 1, 4>;

// Explicit instantiations: every kernel the launchers use is emitted here.
template __global__ void fwd_kernel<BigCfg, false>(FwdParams);
template __global__ void fwd_kernel<SmallCfg, false>(FwdParams);
template __global__ void fwd_kernel<BigCfg, true>(FwdParams);
template __global__ void fwd_kernel<SmallGatedCfg, true>(FwdParams);
template __global__ void dx_kernel<DxCfg>(DxParams);
template __global__ void dx_kernel<DxQuadCfg>(DxParams);
template __global__ void dx_kernel<DxSmallCfg>(DxParams);
template __global__ void dw_kernel<DwCfg, false, false>(DwParams);
template __global__ void dw_kernel<DwCfg, true, false>(DwParams);
template __global__ void dw_kernel<DwCfg, false, true>(DwParams);

// ---------------------------------------------------------------------------
// dW for short reductions (a decode step: a few hundred slots spread over
// many experts, most of them a handful of rows).  There the output is all
// that costs (E*N*K*2 bytes against S*(N+K)*2 of operands), and the tile
// engine spends a copy round trip and a 128 KiB LDS staging pass on every
// 256 x 256 tile whatever its reduction length, with one workgroup per CU to
// hide them.  Here every wave owns 64 (N) x 64 (K) output tiles and works
// alone (no workgroup barrier after the expert table):
//   * operands come from global memory straight into MFMA fragments.  Lane
//     l of v_mfma_f32_32x32x16_bf16 needs 8 consecutive reduction rows of one
//     column: 8 two-byte buffer loads per fragment (32 lanes read 64
//     contiguous bytes of one row; rows past the expert read zero), rows
//     gathered under permute_x / permute_y.  The operands are a few MB and
//     stay in L2.
//   * the tile is computed as its transpose (MFMA rows along K), so a lane
//     holds 4 consecutive K values of one N row; it is rounded to bf16 into
//     a wave-private LDS tile and written out as whole 128-byte row segments,
//     8 rows per store instruction (fp32 output is stored from the
//     accumulators, 16 bytes per lane).
//   * an empty expert's tiles are zeros through the same path.
// Tiles are dealt round-robin over the waves (eight per CU).  The stores
// bound it: on the decode step the same launch with every expert empty (no
// loads, no MFMAs) takes as long as the real one.
constexpr int kSdwWaves = 4;  // waves per workgroup
constexpr int kSdwT = 64;     // output tile: kSdwT rows of N by kSdwT columns of K
constexpr uint32_t kSdwOOB = 1u << 30;
typedef unsigned short u16x8_t __attribute__((ext_vector_type(8)));

template <bool PX, bool PY>
__global__ __launch_bounds__(kSdwWaves * kWave) void dw_small_kernel(DwParams a)
{
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_scratch[2];
    __shared__ __attribute__((aligned(16))) char s_out[kSdwWaves][kSdwT * kSdwT * 2];
    static_assert(sizeof(s_out) >= (kMaxExperts + 1) * sizeof(int), "tile table fits");
    // The table's tile starts are not used here: they go to the output tiles'
    // LDS (four workgroups per CU fit), which the barrier at its end frees.
    build_expert_tables(a.m_sizes, a.E, a.S, s_roff, reinterpret_cast<int *>(&s_out[0][0]),
                        s_scratch, a.err, [](int) { return 0; });
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int col = lane & 31, half = lane >> 5;
    const int ntn = (a.N + kSdwT - 1) / kSdwT, ntk = (a.K + kSdwT - 1) / kSdwT;
    const int per_expert = ntn * ntk;
    const int64_t total = (int64_t)per_expert * a.E;
    const bool f32out = a.flags & MOEGG_DW_FP32_OUT;
    // Operands below 1 GiB each (checked on the host): offsets of 1 GiB and
    // above (kSdwOOB, alone or added to a row or column offset) read zero.
    const uint32_t xrow = (uint32_t)a.K * 2, yrow = (uint32_t)a.N * 2;
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(a.X), 0, (int)((PX ? a.S / a.topk : a.S) * xrow), 0x00020000);
    const __amdgpu_buffer_rsrc_t yr =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(a.dY), 0, (int)(a.S * yrow), 0x00020000);
    char *const lds = s_out[wave];
    const uint32_t Su = (uint32_t)a.S;
    bool bad = false;
    // Byte offsets of this lane's 8 reduction rows c0 + 8 * half + i of the
    // expert starting at slot `start`, in X and in dY (kSdwOOB: zeros, past
    // the expert or a bad gather entry).  The gather loads are unconditional,
    // from clamped in-bounds addresses, so all 8 are in flight together.
    auto step_rows = [&](int start, int m_e, int c0, uint32_t (&ox)[8], uint32_t (&oy)[8]) {
        int g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = start + min(c0 + 8 * half + i, m_e - 1);
            g[i] = (PX || PY) ? a.gather[p] : p;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = c0 + 8 * half + i, p = start + m;
            const bool in = m < m_e;
            const bool ok = !(PX || PY) || (uint32_t)g[i] < Su;
            bad |= in && !ok;
            const int rx = !PX ? p : fast_div((uint32_t)g[i], a.topk_div);
            const int ry = !PY ? p : g[i];
            ox[i] = in && (ok || !PX) ? (uint32_t)rx * xrow : kSdwOOB;
            oy[i] = in && (ok || !PY) ? (uint32_t)ry * yrow : kSdwOOB;
        }
    };
    // Fragment of column c (< lim) over the 8 rows at byte offsets off[]:
    // buffer loads, so that an offset past the operand reads zero.
    auto frag = [&](__amdgpu_buffer_rsrc_t r, const uint32_t (&off)[8], int c,
                    int lim) -> bf16x8_t {
        const uint32_t co = c < lim ? (uint32_t)c * 2 : kSdwOOB;
        u16x8_t v;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __builtin_amdgcn_raw_buffer_load_b16(r, off[i] + co, 0, 0);
        return __builtin_bit_cast(bf16x8_t, v);
    };
    // Tiles are dealt out round-robin over the waves (an expert's tiles cost
    // in proportion to its rows, so contiguous runs would leave the waves
    // of a hot expert behind the rest).
    const int64_t nwaves = (int64_t)gridDim.x * kSdwWaves;
    for (int64_t t = (int64_t)xcd_logical_block(blockIdx.x, gridDim.x) * kSdwWaves + wave;
         t < total; t += nwaves) {
        const int e = (int)(t / per_expert), u = (int)(t % per_expert);
        const int n0 = (u / ntk) * kSdwT, k0 = (u % ntk) * kSdwT;
        const int start = s_roff[e], m_e = s_roff[e + 1] - start;
        f32x16_t acc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = 0.0f;
        for (int c0 = 0; c0 < m_e; c0 += 16) {
            uint32_t ox[8], oy[8];
            step_rows(start, m_e, c0, ox, oy);
            bf16x8_t fa[2], fb[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                fa[j] = frag(xr, ox, k0 + 32 * j + col, a.K);
                fb[j] = frag(yr, oy, n0 + 32 * j + col, a.N);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j],
                                                                         0, 0, 0);
        }
        // acc[i][j][r]: K column k0 + 32 i + 8 (r / 4) + 4 half + r % 4 of
        // N row n0 + 32 j + col.
        if (f32out) {
            float *const out = reinterpret_cast<float *>(a.dW);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int n = n0 + 32 * j + col, k = k0 + 32 * i + 8 * g + 4 * half;
                        if (n < a.N && k < a.K) {
                            const float4 v = {acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                              acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                            *reinterpret_cast<float4 *>(out + ((int64_t)e * a.N + n) * a.K + k) = v;
                        }
                    }
            continue;
        }
        wait_lds();  // the previous tile's reads of this wave's LDS tile are done
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int row = 32 * j + col;
                    const uint2 v = {pack_bf16x2(acc[i][j][4 * g], acc[i][j][4 * g + 1]),
                                     pack_bf16x2(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])};
                    *reinterpret_cast<uint2 *>(lds + row * (kSdwT * 2) +
                                               swz_chunk(row, 4 * i + g) * 16 + half * 8) = v;
                }
        wait_lds();  // every lane's writes are in LDS before any lane reads them
        char *const base = a.dW + (((int64_t)e * a.N + n0) * a.K + k0) * 2;
#pragma unroll
        for (int q = 0; q < kSdwT * kSdwT * 2 / 16 / kWave; ++q) {
            const int idx = q * kWave + lane;
            const int row = idx / 8, c = idx % 8;
            const u32x4_nt_t v = *reinterpret_cast<const u32x4_nt_t *>(
                lds + row * (kSdwT * 2) + swz_chunk(row, c) * 16);
            if (n0 + row < a.N && k0 + 8 * c < a.K)
                __builtin_nontemporal_store(
                    v, reinterpret_cast<u32x4_nt_t *>(base + ((int64_t)row * a.K + 8 * c) * 2));
        }
    }
    if (bad)
        raise_error(a.err, kErrGather);
}
template __global__ void dw_small_kernel<false, false>(DwParams);
template __global__ void dw_small_kernel<true, false>(DwParams);
template __global__ void dw_small_kernel<false, true>(DwParams);
template __global__ void groups_kernel<GroupCfg, true>(GroupsParams);
template __global__ void groups_kernel<GroupCfg, false>(GroupsParams);

static int64_t n_blocks_bound(int64_t rows, int E, int block)
{
    if (rows <= E)
        return rows;
    return (rows - E + 1 + block - 1) / block + E - 1;
}

template <class Kern>
static int resident_blocks(Kern kernel, int threads)
{
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != hipSuccess || n < 1)
        n = 1;
    return n;
}

static int grid_for(int64_t tiles_bound, int cus, int resident)
{
    int64_t g = (int64_t)cus * resident;
    if (tiles_bound < g)
        g = tiles_bound;
    return (int)(g < 1 ? 1 : g);
}

template <class C, bool GATED>
static void fwd_launch_cfg(const FwdParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = n_blocks_bound(p.S, p.E, C::BM) * ((p.N + C::BN - 1) / C::BN);
    static int res = resident_blocks(fwd_kernel<C, GATED>, C::NT);
    hipLaunchKernelGGL((fwd_kernel<C, GATED>), dim3(grid_for(tiles, cus, res)), dim3(C::NT), 0,
                       stream, p);
}

hipError_t fwd_launch(const FwdParams &p, int cus, hipStream_t stream)
{
    const bool small = p.S / p.E < 96;
    if (p.flags & MOEGG_GATED_SILU) {
        if (small)
            fwd_launch_cfg<SmallGatedCfg, true>(p, cus, stream);
        else
            fwd_launch_cfg<BigCfg, true>(p, cus, stream);
    } else {
        if (small)
            fwd_launch_cfg<SmallCfg, false>(p, cus, stream);
        else
            fwd_launch_cfg<BigCfg, false>(p, cus, stream);
    }
    return hipGetLastError();
}

template <class C>
static int dx_resident()
{
    static int res = resident_blocks(dx_kernel<C>, C::NT);
    return res;
}

template <class C>
static void dx_launch_cfg(const DxParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = n_blocks_bound(p.S, p.E, C::BM) * ((p.K + C::BN - 1) / C::BN);
    hipLaunchKernelGGL(dx_kernel<C>, dim3(grid_for(tiles, cus, dx_resident<C>())), dim3(C::NT), 0,
                       stream, p);
    if (p.ws) {
        TailReduceParams r;
        r.ws = p.ws;
        r.out = p.dX;
        r.gather = p.gather;
        r.S = p.S;
        r.ldo = p.K;
        r.ncols = p.K;
        r.scatter_out = p.flags & MOEGG_PERMUTE_X;
        hipLaunchKernelGGL((tail_reduce_kernel<C::BM, C::BN>), dim3(cus * 4), dim3(256), 0, stream,
                           r);
    }
}

// Measured on MI355X: the four-wave engine is faster once the reduction (N)
// is long enough to amortise its per-tile prologue (T=4096 top-2, N=28672:
// 2.16 ms against 2.44 ms); at N = 2048 the eight-wave engine is.
constexpr int kDxQuadMinN = 8192;

// Average rows per expert below which dX uses the small-M tiles: the
// weights are then streamed once per 32-row tile (a decode slice), where
// 256 x 256 tiles would leave about one long, latency-bound tile per CU
// (T=64 top-8 of E=128, N=2048, K=768: 0.064 ms against 0.114 ms).
constexpr int64_t kSmallRows = 96;

// Workspace of the tail split: the header and at most G partials of one
// tile (R * P <= G), for the grid the launch below will use.
template <class C>
static int64_t dx_ws_cfg(int cus)
{
    const int64_t G = (int64_t)cus * dx_resident<C>();
    return G > kTailMaxTiles ? 0 : tail_header_bytes() + G * C::BM * C::BN * 4;
}

// The small-M tiles are many and short (a decode slice): their last round
// costs little, and the finishing launch would cost more.
int64_t dx_workspace_bytes(int64_t S, int E, int N, int K, int cus)
{
    (void)K;
    if (S / E < kSmallRows)
        return 0;
    if (N >= kDxQuadMinN)
        return dx_ws_cfg<DxQuadCfg>(cus);
    return dx_ws_cfg<DxCfg>(cus);
}

hipError_t dx_launch(const DxParams &p, int cus, hipStream_t stream)
{
    if (p.S / p.E < kSmallRows)
        dx_launch_cfg<DxSmallCfg>(p, cus, stream);
    else if (p.N >= kDxQuadMinN)
        dx_launch_cfg<DxQuadCfg>(p, cus, stream);
    else
        dx_launch_cfg<DxCfg>(p, cus, stream);
    return hipGetLastError();
}

// Split reductions.  The target is about three work items per workgroup of
// a full 256-CU chip when the rows are spread evenly over the experts:
// chunks of S * tiles_per_expert / (256 * 3) rows (at least 4 reduction
// steps), so that with the longest items scheduled first no workgroup is
// left with one hot expert's whole reduction.  An expert splits only if it
// has more rows than that; a split expert has fewer than 2 m / split_rows
// chunks, so all of them together hold fewer than 2 S / split_rows partials.
constexpr int kSplitCus = 256, kSplitItems = 3;
constexpr int64_t kNoSplitRows = 1024;

int dw_split_rows(int64_t S, int N, int K)
{
    using C = DwCfg;
    // A launch this short has no reduction long enough to be worth cutting
    // (at most four chunks of 256 rows); without a split the reduce launch
    // is not needed either (a decode step's dW: 4.4 us saved).
    if (S <= kNoSplitRows)
        return 0;
    const int64_t tiles = (int64_t)((N + C::BM - 1) / C::BM) * ((K + C::BN - 1) / C::BN);
    int64_t rows = (S * tiles + kSplitCus * kSplitItems - 1) / (kSplitCus * kSplitItems);
    rows = (rows + BK - 1) / BK * BK;
    if (rows < 4 * BK)
        rows = 4 * BK;
    return rows >= S ? 0 : (int)rows;
}

int64_t dw_workspace_bytes(int64_t S, int E, int N, int K)
{
    const int rows = dw_split_rows(S, N, K);
    if (rows == 0)
        return 0;
    const int64_t partials = 2 * S / rows;
    return dw_header_bytes(E) + partials * N * K * 4;
}

// Byte offset of the gathered X rows in dW's workspace, after the split
// partials.
int64_t dw_gather_offset(int64_t S, int E, int N, int K)
{
    return (dw_workspace_bytes(S, E, N, K) + 255) / 256 * 256;
}

// X rows in expert order for dW under permute_x, when the caller's
// workspace has room for them: xg[p, :] = X[gather[p] / topk, :].  The
// reduction then reads xg in sorted order.  On the Mixtral shape (8192 slots,
// K 4096) the copy takes 0.020 ms and dW 2.00-2.05 ms, against 2.17-2.20 ms
// for the row gather inside dW, with the same result bit for bit: the
// scattered row reads cost dW's copy path more than one streaming pass
// costs.  One workgroup per row at a time; an entry outside [0, S) gives a
// zero row and is reported, as the gather inside dW does.  Only the
// positions the reduction reads are copied: those below the sum of m_sizes
// (negative sizes as 0, clipped to S, as the reduction's tables take them),
// so the entries routing leaves at -1 for dropped slots are not touched.
// Plain stores: dW reads the copy right after.
__global__ __launch_bounds__(256) void gather_x_kernel(DwParams a)
{
    __shared__ long long s_part[256 / kWave];
    long long part = 0;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        part += max(a.m_sizes[e], 0);
    for (int d = kWave / 2; d > 0; d >>= 1)
        part += __shfl_xor(part, d, kWave);
    if ((threadIdx.x & (kWave - 1)) == 0)
        s_part[threadIdx.x / kWave] = part;
    __syncthreads();
    int64_t rows = 0;
    for (int w = 0; w < (int)(blockDim.x / kWave); ++w)
        rows += s_part[w];
    rows = min(rows, a.S);
    const int cpr = a.K / 8;  // 16-byte chunks per row
    for (int64_t p = blockIdx.x; p < rows; p += gridDim.x) {
        const int g = __builtin_amdgcn_readfirstlane(a.gather[p]);
        const bool ok = g >= 0 && g < a.S;
        if (!ok && threadIdx.x == 0)
            raise_error(a.err, kErrGather);
        const char *src = a.X + (int64_t)(ok ? g / a.topk : 0) * a.K * 2;
        char *dst = a.xg + p * a.K * 2;
        for (int c = threadIdx.x; c < cpr; c += blockDim.x)
            *reinterpret_cast<uint4 *>(dst + c * 16) =
                ok ? *reinterpret_cast<const uint4 *>(src + c * 16) : uint4{0, 0, 0, 0};
    }
}

template <bool PX, bool PY>
static void dw_launch_flags(const DwParams &p, int cus, hipStream_t stream)
{
    using C = DwCfg;
    // Work items: every (expert, output tile) plus the extra chunks of split
    // experts, fewer than 2 S / split_rows in all.
    const int64_t per_expert = (int64_t)((p.N + C::BM - 1) / C::BM) * ((p.K + C::BN - 1) / C::BN);
    int64_t tiles = p.E * per_expert;
    if (p.split_rows > 0)
        tiles += 2 * p.S / p.split_rows * per_expert;
    static int res = resident_blocks(dw_kernel<C, PX, PY>, C::NT);
    hipLaunchKernelGGL((dw_kernel<C, PX, PY>), dim3(grid_for(tiles, cus, res)), dim3(C::NT), 0,
                       stream, p);
}


// Launches of at most 1024 slots and at most 16 rows per expert on average
// take dw_small_kernel (no split, no gather copy: the rows are gathered as
// the fragments are loaded).  Measured on MI355X, 128 experts of 2048 x 768:
// a 64-token top-8 decode step (512 slots) 0.092 -> 0.080 ms; 64 experts of
// 2048 x 1408, 512 slots 0.082 -> 0.071 ms; 64 experts of 2048 x 768, 1024
// slots 0.052 -> 0.049 ms.  With 128 rows per expert (8 experts of
// 4096 x 4096, 1024 slots) it is 2.3x slower than the tile engine, whose
// cost does not grow with the reduction here.
constexpr int64_t kSmallDwSlots = 1024, kSmallDwRowsPerExpert = 16;

bool dw_short_launch(int64_t S, int64_t x_rows, int E, int N, int K)
{
    return S <= kSmallDwSlots && S <= kSmallDwRowsPerExpert * E &&
           S * N * 2 < (int64_t)kSdwOOB && x_rows * K * 2 < (int64_t)kSdwOOB;
}

template <bool PX, bool PY>
static void dw_small_launch(const DwParams &p, int cus, hipStream_t stream)
{
    const int64_t tiles = (int64_t)p.E * ((p.N + kSdwT - 1) / kSdwT) * ((p.K + kSdwT - 1) / kSdwT);
    static int res = resident_blocks(dw_small_kernel<PX, PY>, kSdwWaves * kWave);
    hipLaunchKernelGGL((dw_small_kernel<PX, PY>),
                       dim3(grid_for((tiles + kSdwWaves - 1) / kSdwWaves, cus, res)),
                       dim3(kSdwWaves * kWave), 0, stream, p);
}

hipError_t dw_launch(const DwParams &pin, int cus, hipStream_t stream)
{
    DwParams p = pin;
    if (dw_short_launch(p.S, (p.flags & MOEGG_PERMUTE_X) ? p.S / p.topk : p.S, p.E, p.N, p.K)) {
        if (p.flags & MOEGG_PERMUTE_X)
            dw_small_launch<true, false>(p, cus, stream);
        else if (p.flags & MOEGG_PERMUTE_Y)
            dw_small_launch<false, true>(p, cus, stream);
        else
            dw_small_launch<false, false>(p, cus, stream);
        return hipGetLastError();
    }
    if (p.xg && (p.flags & MOEGG_PERMUTE_X) && p.S > 0) {
        hipLaunchKernelGGL(gather_x_kernel, dim3((unsigned)std::min<int64_t>(p.S, (int64_t)cus * 16)),
                           dim3(256), 0, stream, p);
        p.X = p.xg;
        p.flags &= ~MOEGG_PERMUTE_X;
    }
    if (p.flags & MOEGG_PERMUTE_X)
        dw_launch_flags<true, false>(p, cus, stream);
    else if (p.flags & MOEGG_PERMUTE_Y)
        dw_launch_flags<false, true>(p, cus, stream);
    else
        dw_launch_flags<false, false>(p, cus, stream);
    if (p.split_rows > 0 && p.ws)
        hipLaunchKernelGGL(dw_reduce_kernel, dim3(cus * 8), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t groups_launch(const GroupsParams &p, int trans_b, int cus, hipStream_t stream)
{
    using C = GroupCfg;
    int64_t tiles = 0;
    for (int i = 0; i < p.num; ++i)
        tiles += (int64_t)((p.g[i].m + C::BM - 1) / C::BM) * ((p.g[i].n + C::BN - 1) / C::BN);
    if (trans_b) {
        static int res = resident_blocks(groups_kernel<C, true>, C::NT);
        hipLaunchKernelGGL((groups_kernel<C, true>), dim3(grid_for(tiles, cus, res)), dim3(C::NT),
                           0, stream, p);
    } else {
        static int res = resident_blocks(groups_kernel<C, false>, C::NT);
        hipLaunchKernelGGL((groups_kernel<C, false>), dim3(grid_for(tiles, cus, res)), dim3(C::NT),
                           0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace moegg
