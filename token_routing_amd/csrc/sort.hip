// Token rows out to expert order and back, with weights, and the gradients of
// both, gfx950.  Two kernels cover the four operators:
//
//   spread   dst[row(s)] = w[s] * src[t]              (permute; unpermute's dY)
//            dw[s] = <src[t], other[row(s)]>          (unpermute's dw)
//   collect  out[t] = base[t] + sum_j w[s] * in[row(s)]  (unpermute; permute's dX)
//            dw[s] = <other[t], in[row(s)]>           (permute's dw)
//
// for slot s = t * k + j.  Both go by token: the token's row is read (or
// written) once and stays in registers while its k expert-ordered rows pass,
// so every byte moves once and HBM bandwidth is the bound.  WPR waves share a
// token's row; each lane moves 16 bytes at a time.  Sums run in fp32, j
// ascending; a value is rounded once, when it is stored.
//
// In the padded layout every expert's rows are padded to a multiple of
// block_m; spread then also computes row(s) from the unpadded order (the
// slot's expert is the last one whose offset is not above its position) and
// clears the pad rows with workgroups past the tokens'.
#include "elems.h"

#include "layer_params.h"

namespace moegg {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kGroup = 8;  // slots of a token handled together

__device__ __forceinline__ float lanes_sum64(float v)
{
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1)
        v += __shfl_xor(v, d, kWave);
    return v;
}

// dot[j] summed over the lanes of the WPR waves of a token; slot j0 + j's sum
// goes to dw.  Called by every wave of the workgroup together.
template <int WPR>
__device__ __forceinline__ void store_dots(const float (&dot)[kGroup], float *dw, int64_t s0,
                                           int n, bool live, float (*s_dot)[kGroup])
{
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    float sum[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
        sum[j] = lanes_sum64(dot[j]);
    if constexpr (WPR > 1) {
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                s_dot[wave][j] = sum[j];
        __syncthreads();
        if (wave % WPR == 0 && lane < n && live) {
            float total = 0.0f;
            for (int i = 0; i < WPR; ++i)
                total += s_dot[wave + i][lane];
            dw[s0 + lane] = total;
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (lane == 0 && live && j < n)
                dw[s0 + j] = sum[j];
    }
}

template <int DT, bool DOTS, int WPR>
__global__ __launch_bounds__(kSortThreads) void spread_kernel(SpreadParams a, int64_t token_blocks)
{
    typedef typename Elem<DT>::store_t st_t;
    constexpr int P = Elem<DT>::kPer16;
    __shared__ float s_dot[kSortWaves][kGroup];
    st_t *const dst = static_cast<st_t *>(a.dst);

    if ((int64_t)blockIdx.x >= token_blocks) {
        // Pad rows of expert e, dealt out over its pad_blocks workgroups.
        const int b = (int)(blockIdx.x - token_blocks);
        const int e = b / a.pad_blocks;
        const int64_t used = (int64_t)a.offsets[e + 1] - a.offsets[e];
        const int64_t lo = (int64_t)a.padded[e] + (used > 0 ? used : 0);
        const int64_t hi = a.padded[e + 1];
        if (threadIdx.x == 0 && (hi > a.rows || a.padded[e] < 0))
            raise_error(a.err, kErrGather);
        const float zero[P] = {};
        for (int64_t r = (lo > 0 ? lo : 0) + b % a.pad_blocks; r < hi && r < a.rows;
             r += a.pad_blocks)
            for (int col = threadIdx.x * P; col < a.K; col += kSortThreads * P)
                store16<DT>(dst + r * a.K, col, a.K, zero);
        return;
    }

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * (kSortWaves / WPR) + wave / WPR;
    const bool live = t < a.T;
    const st_t *const src = static_cast<const st_t *>(a.src) + t * a.K;
    const st_t *const other = static_cast<const st_t *>(a.other);

    for (int j0 = 0; j0 < a.topk; j0 += kGroup) {
        const int n = min(kGroup, a.topk - j0);
        const int64_t s0 = t * a.topk + j0;
        // Lane j holds slot j's place and weight.
        int place = -1;
        float weight = 1.0f;
        if (live && lane < n) {
            place = a.map[s0 + lane];
            if (a.weights)
                weight = a.weights[s0 + lane];
        }
        if (a.padded && !a.map_is_padded) {
            int count[kGroup] = {};
            for (int e0 = 0; e0 < a.E; e0 += kWave) {
                const int off = e0 + lane < a.E ? a.offsets[e0 + lane] : 0x7fffffff;
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    count[j] += __popcll(__ballot(off <= __shfl(place, j, kWave)));
            }
            int e = 0;
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                e = lane == j ? count[j] - 1 : e;
            if (place >= 0 && lane < n) {
                e = min(max(e, 0), a.E - 1);
                const int64_t to = (int64_t)place + a.padded[e] - a.offsets[e];
                place = to >= 0 && to <= INT32_MAX ? (int)to : INT32_MAX;
            }
        }
        if (place >= a.rows) {
            raise_error(a.err, kErrGather);
            place = -1;
        }
        if (a.row_map && live && lane < n && wave % WPR == 0)
            a.row_map[s0 + lane] = place;
        int row[kGroup];
        float w[kGroup], dot[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            row[j] = __builtin_amdgcn_readlane(place, j);
            w[j] = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j));
            dot[j] = 0.0f;
        }
        if (live)
            for (int c0 = (wave % WPR) * kWave * P; c0 < a.K; c0 += WPR * kWave * P) {
                const int col = c0 + lane * P;
                float x[P];
                widen_all<DT>(x, load16<DT>(src, col, a.K));
                if constexpr (DOTS) {
                    typename Pack16<DT>::vec_t raw[kGroup];
#pragma unroll
                    for (int j = 0; j < kGroup; ++j)
                        if (row[j] >= 0)
                            raw[j] = load16<DT>(other + (int64_t)row[j] * a.K, col, a.K);
#pragma unroll
                    for (int j = 0; j < kGroup; ++j)
                        if (row[j] >= 0) {
                            float y[P];
                            widen_all<DT>(y, raw[j]);
#pragma unroll
                            for (int i = 0; i < P; ++i)
                                dot[j] += x[i] * y[i];
                        }
                }
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    if (row[j] >= 0) {
                        float v[P];
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            v[i] = w[j] * x[i];
                        store16<DT>(dst + (int64_t)row[j] * a.K, col, a.K, v);
                    }
            }
        if constexpr (DOTS)
            store_dots<WPR>(dot, a.dw, s0, n, live, s_dot);
    }
}

template <int DT, bool DOTS, int WPR>
__global__ __launch_bounds__(kSortThreads) void collect_kernel(CollectParams a)
{
    typedef typename Elem<DT>::store_t st_t;
    typedef typename Pack16<DT>::vec_t vec_t;
    constexpr int P = Elem<DT>::kPer16;
    __shared__ float s_dot[kSortWaves][kGroup];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * (kSortWaves / WPR) + wave / WPR;
    const bool live = t < a.T;
    const st_t *const in = static_cast<const st_t *>(a.rows_in);
    const st_t *const base = static_cast<const st_t *>(a.base) + t * a.K;
    const st_t *const other = static_cast<const st_t *>(a.other) + t * a.K;
    st_t *const out = static_cast<st_t *>(a.out) + t * a.K;
    const int first = (wave % WPR) * kWave * P;

    int row[kGroup];
    float w[kGroup], dot[kGroup];
    // Slots [j0, j0 + 8) of the token: their rows and weights, the same in
    // every lane.  Lane j loads slot j's, so every lane of the wave has to be
    // here: the column loops run on a column that is the same for the wave,
    // and lanes past the row's end load and store nothing.
    auto fetch = [&](int j0) {
        int place = -1;
        float weight = 1.0f;
        if (live && lane < min(kGroup, a.topk - j0)) {
            const int64_t s = t * a.topk + j0 + lane;
            place = a.map[s];
            if (a.weights)
                weight = a.weights[s];
            if (place >= a.rows) {
                raise_error(a.err, kErrGather);
                place = -1;
            }
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            row[j] = __builtin_amdgcn_readlane(place, j);
            w[j] = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j));
            dot[j] = 0.0f;
        }
    };
    auto load_rows = [&](vec_t (&raw)[kGroup], int col) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (row[j] >= 0)
                raw[j] = load16<DT>(in + (int64_t)row[j] * a.K, col, a.K);
    };
    auto add_dots = [&](const vec_t (&raw)[kGroup], int col) {
        float x[P];
        widen_all<DT>(x, load16<DT>(other, col, a.K));
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (row[j] >= 0) {
                float y[P];
                widen_all<DT>(y, raw[j]);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    dot[j] += x[i] * y[i];
            }
    };

    // More slots than the registers hold at once: their dots in a pass of their
    // own, ahead of the stores, since out may be `other`.
    if constexpr (DOTS)
        if (a.topk > kGroup)
            for (int j0 = 0; j0 < a.topk; j0 += kGroup) {
                fetch(j0);
                if (live)
                    for (int c0 = first; c0 < a.K; c0 += WPR * kWave * P) {
                        vec_t raw[kGroup];
                        load_rows(raw, c0 + lane * P);
                        add_dots(raw, c0 + lane * P);
                    }
                store_dots<WPR>(dot, a.dw, t * a.topk + j0, min(kGroup, a.topk - j0), live, s_dot);
            }
    fetch(0);
    if (live)
        for (int c0 = first; c0 < a.K; c0 += WPR * kWave * P) {
            const int col = c0 + lane * P;
            float acc[P];
            if (a.base) {
                widen_all<DT>(acc, load16<DT>(base, col, a.K));
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    acc[i] = 0.0f;
            }
            for (int j0 = 0; j0 < a.topk; j0 += kGroup) {
                if (a.topk > kGroup)
                    fetch(j0);
                vec_t raw[kGroup];
                load_rows(raw, col);
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    if (row[j] >= 0) {
                        float y[P];
                        widen_all<DT>(y, raw[j]);
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            acc[i] += w[j] * y[i];
                    }
                if constexpr (DOTS)
                    if (a.topk <= kGroup)
                        add_dots(raw, col);
            }
            store16<DT>(out, col, a.K, acc);
        }
    if constexpr (DOTS)
        if (a.topk <= kGroup)
            store_dots<WPR>(dot, a.dw, t * a.topk, a.topk, live, s_dot);
}

// Waves that share a token's row: as many (1, 2 or 4) as it fills with 16
// bytes a lane.
inline int waves_per_row(int K, int per16)
{
    const int chunks = (K + kWave * per16 - 1) / (kWave * per16);
    return chunks >= 4 ? 4 : chunks >= 2 ? 2 : 1;
}

template <int DT, bool DOTS, int WPR>
hipError_t spread_go(const SpreadParams &p, hipStream_t stream)
{
    const int64_t tb = (p.T + kSortWaves / WPR - 1) / (kSortWaves / WPR);
    const int64_t grid = tb + (p.padded ? (int64_t)p.E * p.pad_blocks : 0);
    hipLaunchKernelGGL((spread_kernel<DT, DOTS, WPR>), dim3((unsigned)grid), dim3(kSortThreads), 0,
                       stream, p, tb);
    return hipGetLastError();
}

template <int DT, bool DOTS> hipError_t spread_wpr(const SpreadParams &p, hipStream_t stream)
{
    switch (waves_per_row(p.K, Elem<DT>::kPer16)) {
    case 4: return spread_go<DT, DOTS, 4>(p, stream);
    case 2: return spread_go<DT, DOTS, 2>(p, stream);
    default: return spread_go<DT, DOTS, 1>(p, stream);
    }
}

template <int DT> hipError_t spread_dt(const SpreadParams &p, hipStream_t stream)
{
    return p.dw ? spread_wpr<DT, true>(p, stream) : spread_wpr<DT, false>(p, stream);
}

template <int DT, bool DOTS, int WPR>
hipError_t collect_go(const CollectParams &p, hipStream_t stream)
{
    const int64_t tb = (p.T + kSortWaves / WPR - 1) / (kSortWaves / WPR);
    hipLaunchKernelGGL((collect_kernel<DT, DOTS, WPR>), dim3((unsigned)tb), dim3(kSortThreads), 0,
                       stream, p);
    return hipGetLastError();
}

template <int DT, bool DOTS> hipError_t collect_wpr(const CollectParams &p, hipStream_t stream)
{
    switch (waves_per_row(p.K, Elem<DT>::kPer16)) {
    case 4: return collect_go<DT, DOTS, 4>(p, stream);
    case 2: return collect_go<DT, DOTS, 2>(p, stream);
    default: return collect_go<DT, DOTS, 1>(p, stream);
    }
}

template <int DT> hipError_t collect_dt(const CollectParams &p, hipStream_t stream)
{
    return p.dw ? collect_wpr<DT, true>(p, stream) : collect_wpr<DT, false>(p, stream);
}

}  // namespace

hipError_t spread_launch(const SpreadParams &p0, int dtype, hipStream_t stream)
{
    if (p0.T == 0 && !p0.padded)
        return hipSuccess;
    SpreadParams p = p0;
    // About a thousand workgroups clear pad rows, whatever the number of experts.
    p.pad_blocks = p.E > 0 ? (p.E >= 1024 ? 1 : p.E <= 16 ? 64 : 1024 / p.E) : 1;
    return dtype == kBf16   ? spread_dt<kBf16>(p, stream)
           : dtype == kFp16 ? spread_dt<kFp16>(p, stream)
                            : spread_dt<kFp32>(p, stream);
}

hipError_t collect_launch(const CollectParams &p, int dtype, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    return dtype == kBf16   ? collect_dt<kBf16>(p, stream)
           : dtype == kFp16 ? collect_dt<kFp16>(p, stream)
                            : collect_dt<kFp32>(p, stream);
}

}  // namespace moegg
