// 8-bit forms of activations, gfx950: rows of int8 with one scale (quant_rows),
// packed blocks (pack8, unpack8, and unpack_rows: packed rows in expert order), and
// rows copied to whole 16-byte chunks (pad_rows).  All are streams over their
// bytes; a lane moves 16 bytes of values at a time.
#include "elems.h"

#include "block_params.h"
#include "pack.h"

namespace moegg {

namespace {

constexpr int kPackThreads = 256;

// 8 values of a row of n elements (zeros at and past n), in fp32.
template <int DT>
__device__ __forceinline__ void load8f(const typename Elem<DT>::store_t *row, int col, int n,
                                       float (&f)[8])
{
    if constexpr (DT == kFp32) {
        const auto a = load16<DT>(row, col, n), b = load16<DT>(row, col + 4, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    } else {
        widen_all<DT>(f, load16<DT>(row, col, n));
    }
}

template <int DT>
__device__ __forceinline__ void store8f(typename Elem<DT>::store_t *row, int col, int n,
                                        const float (&f)[8])
{
    store16<DT, false>(row, col, n, f);
    if constexpr (DT == kFp32)
        store16<DT, false>(row, col + 4, n, f + 4);
}

// Largest of the lanes' values over groups of 4 neighbours.
__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m)
{
    for (int d = 1; d < kWave; d <<= 1)
        m = max(m, (uint32_t)__shfl_xor((int)m, d, kWave));
    return m;
}

// round(127 x / m) of real numbers, ties to even.  t = x * (127 / m) is within
// 2^-23 * 127 of the quotient; where that leaves the rounding open, the quotient
// is taken in 64 bits: 127 x is exact there (31 bits), and a quotient of at least
// 1/2 by a number of 24 bits is either a tie or at least 2^-34 away from one.
__device__ __forceinline__ int row_code(float x, float inv, float m)
{
    const float t = x * inv;
    const float r = rintf(t);
    if (fabsf(fabsf(t - r) - 0.5f) < 1e-4f)
        return (int)rint((double)x * 127.0 / (double)m);
    return (int)r;
}

}  // namespace

// One workgroup of THREADS per row.  A row's values stay in registers between
// the maximum and the codes up to THREADS * 32 columns; the columns past that
// are read again.
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS) void quant_rows_kernel(QuantParams a)
{
    typedef typename Elem<DT>::store_t T;
    constexpr int PER = 4;
    __shared__ uint32_t s_max[THREADS / kWave];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    char *q = a.Q + row * a.Kq;
    float f[PER][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = (i * THREADS + (int)threadIdx.x) * 8;
        if (col < a.K) {
            load8f<DT>(x, col, a.K, f[i]);
            m = max(m, abs_max_bits(f[i]));
        }
    }
    for (int col = (PER * THREADS + (int)threadIdx.x) * 8; col < a.K; col += THREADS * 8) {
        float g[8];
        load8f<DT>(x, col, a.K, g);
        m = max(m, abs_max_bits(g));
    }
    m = wave_max(m);
    if constexpr (THREADS > kWave) {
        if (threadIdx.x % kWave == 0)
            s_max[threadIdx.x / kWave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / kWave; ++w)
            m = max(m, s_max[w]);
    }
    const bool finite = m < kInfBits;
    const float top = __builtin_bit_cast(float, m);
    // 127 / m overflows for the smallest subnormals: the codes then come from
    // the 64-bit quotient (t is infinite or NaN, and compares as no tie).
    const float inv = 127.0f / top;
    const bool narrow = !(inv < __builtin_inff());
    if (threadIdx.x == 0)
        a.scales[row] = finite ? top / 127.0f : __builtin_nanf("");
    auto put = [&](int col, const float (&g)[8]) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int c = 0;
            if (finite && m != 0)
                c = narrow ? (int)rint((double)g[i] * 127.0 / (double)top)
                           : row_code(g[i], inv, top);
            w[i / 4] |= (uint32_t)(c & 255) << (8 * (i % 4));
        }
        *reinterpret_cast<uint2 *>(q + col) = uint2{w[0], w[1]};
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = (i * THREADS + (int)threadIdx.x) * 8;
        if (col < a.K)
            put(col, f[i]);
        else if (col < a.Kq)
            *reinterpret_cast<uint2 *>(q + col) = uint2{0, 0};
    }
    for (int col = (PER * THREADS + (int)threadIdx.x) * 8; col < a.Kq; col += THREADS * 8) {
        float g[8] = {};
        if (col < a.K)
            load8f<DT>(x, col, a.K, g);
        put(col, g);
    }
}

// Four lanes per block of 32, 8 columns each.
template <int DT>
__global__ __launch_bounds__(kPackThreads) void pack8_kernel(PackParams a)
{
    typedef typename Elem<DT>::store_t T;
    const int64_t Cp = packed_cols(a.cols);
    const uint32_t cpr = (uint32_t)(Cp / 8);  // chunks of 8 columns per row
    const int64_t total = a.rows * cpr;
    for (int64_t base = (int64_t)blockIdx.x * kPackThreads; base < total;
         base += (int64_t)gridDim.x * kPackThreads) {
        const int64_t r0 = base / cpr;
        const uint32_t in = (uint32_t)(base - r0 * cpr) + threadIdx.x;
        const int64_t row = r0 + in / cpr;
        const int col = (int)(in % cpr) * 8;
        if (row >= a.rows)
            continue;
        float f[8];
        load8f<DT>(static_cast<const T *>(a.X) + row * a.ldx, col, a.cols, f);
        uint32_t b = pack_exp(quad_max(abs_max_bits(f))), w[2];
        pack_codes(f, b, w);
        *reinterpret_cast<uint2 *>(a.Q + row * Cp + col) = uint2{w[0], w[1]};
        if ((threadIdx.x & 3) == 0)
            a.S[(row * Cp + col) / kPackBlock] = (uint8_t)b;
    }
}

// fp16 holds no more than 65504: a step past it is taken there.
template <int DT>
__device__ __forceinline__ float in_range(float f)
{
    return DT == kFp16 && f == f ? fminf(fmaxf(f, -65504.0f), 65504.0f) : f;
}

template <int DT>
__global__ __launch_bounds__(kPackThreads) void unpack8_kernel(PackParams a)
{
    typedef typename Elem<DT>::store_t T;
    const int64_t Cp = packed_cols(a.cols);
    const uint32_t cpr = (uint32_t)((a.cols + 7) / 8);
    const int64_t total = a.rows * cpr;
    for (int64_t base = (int64_t)blockIdx.x * kPackThreads; base < total;
         base += (int64_t)gridDim.x * kPackThreads) {
        const int64_t r0 = base / cpr;
        const uint32_t in = (uint32_t)(base - r0 * cpr) + threadIdx.x;
        const int64_t row = r0 + in / cpr;
        const int col = (int)(in % cpr) * 8;
        if (row >= a.rows)
            continue;
        const uint2 q = *reinterpret_cast<const uint2 *>(a.Q + row * Cp + col);
        const float step = pack_step(a.S[(row * Cp + col) / kPackBlock]);
        float f[8];
        unpack4(q.x, step, f);
        unpack4(q.y, step, f + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = in_range<DT>(f[i]);
        store8f<DT>(static_cast<T *>(a.out) + row * a.ldx, col, a.cols, f);
    }
}

// One workgroup per row at a time; as the copy in front of dW, an entry of
// gather outside [0, rows) gives a zero row and is reported, and only the
// positions below the sum of m_sizes are written.
__global__ __launch_bounds__(kPackThreads) void unpack_rows_kernel(UnpackRowsParams a)
{
    __shared__ long long s_part[kPackThreads / kWave];
    int64_t rows = a.rows;
    if (a.m_sizes) {
        long long part = 0;
        for (int e = threadIdx.x; e < a.E; e += kPackThreads)
            part += max(a.m_sizes[e], 0);
        for (int d = kWave / 2; d > 0; d >>= 1)
            part += __shfl_xor(part, d, kWave);
        if ((threadIdx.x & (kWave - 1)) == 0)
            s_part[threadIdx.x / kWave] = part;
        __syncthreads();
        int64_t sum = 0;
        for (int w = 0; w < kPackThreads / kWave; ++w)
            sum += s_part[w];
        rows = min(rows, sum);
    }
    const int64_t Cp = packed_cols(a.cols);
    for (int64_t p = blockIdx.x; p < rows; p += gridDim.x) {
        int64_t src = p;
        bool ok = true;
        if (a.gather) {
            const int g = __builtin_amdgcn_readfirstlane(a.gather[p]);
            ok = g >= 0 && g < a.rows;
            src = ok ? g / a.topk : 0;
            if (!ok && threadIdx.x == 0)
                raise_error(a.err, kErrGather);
        }
        const char *q = a.Q + src * Cp;
        const uint8_t *s = a.S + src * Cp / kPackBlock;
        uint16_t *out = reinterpret_cast<uint16_t *>(a.out) + p * a.cols;
        for (int col = threadIdx.x * 8; col < a.cols; col += kPackThreads * 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(q + col);
            const float step = pack_step(s[col / kPackBlock]);
            float f[8] = {};
            if (ok) {
                unpack4(v.x, step, f);
                unpack4(v.y, step, f + 4);
            }
            store16<kBf16, false>(out, col, a.cols, f);
        }
    }
}

__global__ __launch_bounds__(kPackThreads) void pad_rows_kernel(PadParams a)
{
    const int cpr = (a.cols + 7) / 8;
    const int64_t total = a.groups * a.rows;
    // Whole groups without rows are passed over; a workgroup takes a row at a time.
    for (int64_t r = blockIdx.x; r < total; r += gridDim.x) {
        if (a.m_sizes && a.m_sizes[r / a.rows] <= 0)
            continue;
        const uint16_t *src = reinterpret_cast<const uint16_t *>(a.src) + r * a.cols;
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.dst) + r * cpr * 8;
        for (int c = threadIdx.x; c < cpr; c += kPackThreads)
            *reinterpret_cast<Pack16<kBf16>::vec_t *>(dst + c * 8) =
                load16<kBf16>(src, c * 8, a.cols);
    }
}

namespace {

unsigned pack_grid(int64_t items)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(items, 256 * 32));
}

template <int DT>
void quant_cfg(const QuantParams &p, hipStream_t stream)
{
    // A wave per row up to the columns it keeps in registers.
    if (p.K <= kWave * 32)
        hipLaunchKernelGGL((quant_rows_kernel<DT, kWave>), dim3((unsigned)p.rows), dim3(kWave), 0,
                           stream, p);
    else
        hipLaunchKernelGGL((quant_rows_kernel<DT, 256>), dim3((unsigned)p.rows), dim3(256), 0,
                           stream, p);
}

}  // namespace

hipError_t quant_rows_launch(const QuantParams &p, int dtype, hipStream_t stream)
{
    if (dtype == kBf16)
        quant_cfg<kBf16>(p, stream);
    else if (dtype == kFp16)
        quant_cfg<kFp16>(p, stream);
    else
        quant_cfg<kFp32>(p, stream);
    return hipGetLastError();
}

hipError_t pack8_launch(const PackParams &p, int dtype, hipStream_t stream)
{
    const int64_t items = (p.rows * (packed_cols(p.cols) / 8) + kPackThreads - 1) / kPackThreads;
    const dim3 grid(pack_grid(items)), block(kPackThreads);
    if (dtype == kBf16)
        hipLaunchKernelGGL(pack8_kernel<kBf16>, grid, block, 0, stream, p);
    else if (dtype == kFp16)
        hipLaunchKernelGGL(pack8_kernel<kFp16>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(pack8_kernel<kFp32>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t unpack8_launch(const PackParams &p, int dtype, hipStream_t stream)
{
    const int64_t items = (p.rows * ((p.cols + 7) / 8) + kPackThreads - 1) / kPackThreads;
    const dim3 grid(pack_grid(items)), block(kPackThreads);
    if (dtype == kBf16)
        hipLaunchKernelGGL(unpack8_kernel<kBf16>, grid, block, 0, stream, p);
    else if (dtype == kFp16)
        hipLaunchKernelGGL(unpack8_kernel<kFp16>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(unpack8_kernel<kFp32>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t unpack_rows_launch(const UnpackRowsParams &p, int cus, hipStream_t stream)
{
    hipLaunchKernelGGL(unpack_rows_kernel,
                       dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(p.rows, cus * 16))),
                       dim3(kPackThreads), 0, stream, p);
    return hipGetLastError();
}

hipError_t pad_rows_launch(const PadParams &p, int cus, hipStream_t stream)
{
    const int64_t rows = p.groups * p.rows;
    hipLaunchKernelGGL(pad_rows_kernel,
                       dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(rows, cus * 16))),
                       dim3(kPackThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace moegg
