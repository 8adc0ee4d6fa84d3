// Y = grouped X W_e^T of a few rows, gfx950: the serving forms (8-bit integers, and the
// gated block in bf16 with nothing kept) of block_fwd.h where experts have one or a few
// rows.
//
// The weights are read once and bound it: a tile of 32 rows gives each of its few
// workgroups a long chain of stages, and too few bytes are on their way.  Here a wave
// owns 4 rows of W and its lanes share the reduction, 16 bytes of each row at a
// time, straight to registers; the products of a lane are summed in it, and the
// lanes' sums by register moves at the end.
#include "block_epilogue.h"

namespace moegg {

namespace {

constexpr int kVecThreads = 256;
constexpr int kVecRows = 4;   // rows of W a wave

template <int CTRL, class T>
__device__ __forceinline__ T add_moved(T v)
{
    const int b = __builtin_bit_cast(int, v);
    return v + __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, b, CTRL, 0xf, 0xf, false));
}

// Sums of four values over the wave: lanes 16 q .. + 15 get value sum_of(q).  Exchanges
// of halves and of rows of 16 lanes fold two values into one register each, then
// the rows are summed by rotations: 10 instructions where four sums apart take 32.
__device__ __forceinline__ int sum_of(int q)
{
    return (q & 1) << 1 | q >> 1;
}
template <class T>
__device__ __forceinline__ T sum4(const T (&v)[4])
{
    T h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v[2 * i]),
                                                        __builtin_bit_cast(uint32_t, v[2 * i + 1]),
                                                        false, false);
        h[i] = __builtin_bit_cast(T, (uint32_t)r[0]) + __builtin_bit_cast(T, (uint32_t)r[1]);
    }
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, h[0]),
                                                    __builtin_bit_cast(uint32_t, h[1]), false, false);
    T t = __builtin_bit_cast(T, (uint32_t)r[0]) + __builtin_bit_cast(T, (uint32_t)r[1]);
    t = add_moved<0x121>(t);
    t = add_moved<0x122>(t);
    t = add_moved<0x124>(t);
    return add_moved<0x128>(t);
}

__device__ __forceinline__ void dot16(const u32x4_t &x, const u32x4_t &w, int &acc)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        acc = __builtin_amdgcn_sdot4((int)x[i], (int)w[i], acc, false);
}
__device__ __forceinline__ void dot16(const u32x4_t &x, const u32x4_t &w, float &acc)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc = __builtin_fmaf(__uint_as_float(x[i] << 16), __uint_as_float(w[i] << 16), acc);
        acc = __builtin_fmaf(__uint_as_float(x[i] & 0xffff0000u),
                             __uint_as_float(w[i] & 0xffff0000u), acc);
    }
}

}  // namespace

// ROWS rows of an expert a workgroup at a time, 4 rows of W a wave: 4 output columns,
// or gate and up of 2.
template <bool I8, int ACT, int ROWS>
__global__ __launch_bounds__(kVecThreads) void block_vec_kernel(BlockFwdParams a)
{
    constexpr bool GATED = ACT != kPlain;
    constexpr int COLS = GATED ? kVecRows / 2 : kVecRows;
    constexpr int WG_COLS = COLS * (kVecThreads / kWave);
    typedef std::conditional_t<I8, int, float> Sum;
    __shared__ int s_roff[kMaxExperts + 1];
    __shared__ int s_tstart[kMaxExperts + 1];
    __shared__ int s_scratch[2];

    const bool px = a.flags & MOEGG_PERMUTE_X, py = a.flags & MOEGG_PERMUTE_Y;
    const bool fm = a.flags & MOEGG_FUSE_MUL_POST;
    const bool halves = a.flags & MOEGG_GATED_HALVES;
    const int cols = GATED ? a.N / 2 : a.N;
    const int ntc = (cols + WG_COLS - 1) / WG_COLS;
    const int total = build_expert_tables(a.m_sizes, a.E, a.S, s_roff, s_tstart, s_scratch, a.err,
                                          [&](int m) { return (m + ROWS - 1) / ROWS * ntc; });
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int bytes = a.K * 2;

    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(upper_index(s_tstart, a.E, t));
        const int r0 = __builtin_amdgcn_readfirstlane(s_roff[e]);
        const int mc = __builtin_amdgcn_readfirstlane(s_roff[e + 1]) - r0;
        const int u = t - __builtin_amdgcn_readfirstlane(s_tstart[e]);
        // An expert's row groups at one set of columns follow each other.
        const int groups = (mc + ROWS - 1) / ROWS;
        const int c0 = u / groups * WG_COLS + wave * COLS;
        const int p0 = r0 + u % groups * ROWS, rows = min(ROWS, mc - u % groups * ROWS);
        if (c0 >= cols)
            continue;

        // Columns past the last one and rows past the last one repeat it.
        const char *w[kVecRows];
        int wrow[kVecRows];
#pragma unroll
        for (int j = 0; j < kVecRows; ++j) {
            const int c = min(c0 + (GATED ? j / 2 : j), cols - 1);
            wrow[j] = !GATED ? c : halves ? c + j % 2 * cols : 2 * c + j % 2;
            w[j] = a.W + ((int64_t)e * a.N + wrow[j]) * a.ldw;
        }
        const char *x[ROWS];
        int src[ROWS], dst[ROWS], slot[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int p = p0 + min(r, rows - 1);
            int g = p;
            if (px || py)
                g = __builtin_amdgcn_readfirstlane(a.gather[p]);
            const bool ok = g >= 0 && g < a.S;
            if (!ok && lane == 0)
                raise_error(a.err, kErrGather);
            slot[r] = ok ? g : 0;
            src[r] = px ? slot[r] / a.topk : p;
            dst[r] = r < rows && ok ? (py ? g : p) : -1;
            x[r] = a.X + src[r] * a.ldx;
        }

        // This lane's row of W: wave sums of four (sum_of).
        const int j = sum_of(lane >> 4);
        float ws = 1.0f;
        if constexpr (I8) {
            int own = wrow[0];
#pragma unroll
            for (int i = 1; i < kVecRows; ++i)
                own = j == i ? wrow[i] : own;
            ws = a.w_scales[(int64_t)e * a.N + own];
        }
        // Lane 16 q + r finishes row r's column.
        float f = 0.0f, v = 0.0f;
        int64_t at = -1;
        auto products = [&](auto count) {
            constexpr int R = decltype(count)::value;
            Sum acc[R][kVecRows] = {};
#pragma unroll 2
            for (int k = lane * 16; k < bytes; k += kWave * 16) {
                u32x4_t xv[R], wv[kVecRows];
#pragma unroll
                for (int i = 0; i < kVecRows; ++i)
                    wv[i] = *reinterpret_cast<const u32x4_t *>(w[i] + k);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    xv[r] = *reinterpret_cast<const u32x4_t *>(x[r] + k);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < kVecRows; ++i)
                        dot16(xv[r], wv[i], acc[r][i]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s = 1.0f;
                if constexpr (I8)
                    s = a.x_scales[src[r]];
                if (fm)
                    s *= a.topk_w[slot[r]];
                float y = (float)sum4(acc[r]) * s * ws, up = 0.0f;
                int c = j;
                if constexpr (GATED) {  // lanes below 32 hold gates, the others their partners
                    uint32_t g = __float_as_uint(y), u = g;
                    swap_halves(g, u);
                    y = __uint_as_float(g);
                    up = __uint_as_float(u);
                    c = lane >> 4 & 1;
                }
                if ((lane & 15) == r && dst[r] >= 0 && c0 + c < cols && (!GATED || lane < 32)) {
                    f = y;
                    v = up;
                    at = (int64_t)dst[r] * cols + c0 + c;
                }
            }
        };
        if (rows == 1)
            products(std::integral_constant<int, 1>{});
        else if constexpr (ROWS > 1) {
            if (rows == 2)
                products(std::integral_constant<int, 2>{});
            else
                products(std::integral_constant<int, ROWS>{});
        }
        if (at >= 0) {
            if constexpr (GATED)
                f = GateAct<ACT == kGelu>::act(f) * v;
            reinterpret_cast<uint16_t *>(a.Y)[at] = (uint16_t)pack_bf16x2(f, f);
        }
    }
}

template <bool I8, int ACT, int ROWS>
static void block_vec_cfg(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    const int cols = ACT == kPlain ? p.N : p.N / 2;
    const int wg_cols = (ACT == kPlain ? kVecRows : kVecRows / 2) * (kVecThreads / kWave);
    const int64_t tiles = row_tiles(p.S, p.E, ROWS) * ((cols + wg_cols - 1) / wg_cols);
    static const int most = resident_workgroups(block_vec_kernel<I8, ACT, ROWS>, kVecThreads);
    const int64_t grid = std::max<int64_t>(1, std::min((int64_t)cus * most, tiles));
    hipLaunchKernelGGL((block_vec_kernel<I8, ACT, ROWS>), dim3((unsigned)grid), dim3(kVecThreads), 0,
                       stream, p);
}

template <bool I8, int ACT>
static void block_vec_rows(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.S <= p.topk)  // one token: one row an expert
        block_vec_cfg<I8, ACT, 1>(p, cus, stream);
    else
        block_vec_cfg<I8, ACT, 4>(p, cus, stream);
}

template <bool I8>
static hipError_t block_vec_act(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (p.flags & MOEGG_GATED_SILU)
        block_vec_rows<I8, kSilu>(p, cus, stream);
    else if (p.flags & MOEGG_GATED_GELU)
        block_vec_rows<I8, kGelu>(p, cus, stream);
    else if constexpr (I8)
        block_vec_rows<I8, kPlain>(p, cus, stream);
    return hipGetLastError();
}

bool block_vec_pays(const BlockFwdParams &p, int cus)
{
    const bool gated = p.flags & (MOEGG_GATED_SILU | MOEGG_GATED_GELU);
    return vec_pays(p.S, p.E, p.N, gated, (int64_t)p.K * 2, cus);
}

hipError_t block_vec_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    return p.w_scales ? block_vec_act<true>(p, cus, stream) : block_vec_act<false>(p, cus, stream);
}

}  // namespace moegg
