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

// Over the wave: rotations inside the rows of 16 lanes, then exchanges of rows and
// halves, registers all (six shuffles through LDS cost 65536 rows 4 us).
__device__ __forceinline__ uint32_t wave_max(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xf, 0xf, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, false));
    const auto r = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(r[0], r[1]);
    const auto h = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(h[0], h[1]);
}

// About 127 / m: v_rcp_f32 is good to an ulp, the product to half a one (where both are
// normal numbers).
__device__ __forceinline__ float row_inverse(uint32_t m)
{
    return 127.0f * __builtin_amdgcn_rcpf(__uint_as_float(m));
}

// round(127 x / m) of real numbers, ties to even, for 8 values, as bytes.  x times a
// number just below 127 / m and x times one just above it (2^-21 beside inv, which is
// within 1.5 * 2^-23) are rounded by adding 1.5 * 2^23 in an fma, which leaves the whole
// number in the low byte: where both give the same, the quotient between them does.
// Else it is so near to a tie that the rounding is open, and the quotients are taken in
// 64 bits, as where inv is no number to use: 127 x is exact there (31 bits), and a
// quotient of at least 1/2 by a number of 24 bits is either a tie or at least 2^-34
// away from one.
__device__ __forceinline__ void row_codes(const float (&x)[8], float inv, float m,
                                          uint32_t (&w)[2])
{
    constexpr float kRound = 12582912.0f, kStep = 0x1p-21f;
    const float lo = inv * (1.0f - kStep), hi = inv * (1.0f + kStep);
    uint32_t c[8], open = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = __float_as_uint(__builtin_fmaf(x[i], lo, kRound));
        open = (c[i] ^ __float_as_uint(__builtin_fmaf(x[i], hi, kRound))) + open;
    }
    if (open != 0 || !(inv > 127.0f * 0x1p-126f && hi < __builtin_inff())) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c[i] = (uint32_t)(int)rint((double)x[i] * 127.0 / (double)m);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0c0c0400u) |
               __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x04000c0cu);
}

// The fp32 bits of the largest magnitude among 8 values as they stand in memory.  16-bit
// types are compared as they are, two at a time.
template <int DT, int V>
__device__ __forceinline__ uint32_t raw_max_bits(const typename Pack16<DT>::vec_t (&v)[V])
{
    if constexpr (DT == kFp32) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                m = max(m, __float_as_uint(v[i][k]) & kAbsBits);
        return m;
    } else {
        typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
        typedef uint32_t words_t __attribute__((ext_vector_type(4)));
        const words_t w = __builtin_bit_cast(words_t, v[0]);
        u16x2_t m = __builtin_bit_cast(u16x2_t, w[0] & 0x7fff7fffu);
#pragma unroll
        for (int k = 1; k < 4; ++k)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[k] & 0x7fff7fffu));
        return __float_as_uint(Elem<DT>::widen(max(m[0], m[1])));
    }
}

}  // namespace

// The codes of a row's columns col .. col + 7 (m: the bits of its largest value, inv
// about 127 / m); a row of zeros, or one that is not finite, has codes 0.
__device__ __forceinline__ void put_codes(char *q, int col, const float (&g)[8], uint32_t m,
                                          float inv)
{
    uint32_t w[2] = {0, 0};
    if (m - 1u < kInfBits - 1u)
        row_codes(g, inv, __uint_as_float(m), w);
    *reinterpret_cast<uint2 *>(q + col) = uint2{w[0], w[1]};
}
__device__ __forceinline__ float row_scale(uint32_t m)
{
    return m < kInfBits ? __uint_as_float(m) / 127.0f : __builtin_nanf("");
}

// Rows of up to PER * 512 columns: a wave for each.  TAIL: K is not a multiple of 8.
// 65536 rows of bf16: of 768 40 us (3.8 TB/s read and written, where a row costs as much as
// one of 1024), of 1024 43 (4.7), of 512 26.8 (3.8); a token of 1024 2.3 us, the launch.
// Slower: waves that go on to further rows, their loads ahead (44.0, 48.3, 34.8: they wait for
// their stores as well); two or four rows loaded together (41.7, 44.8, 25.8 and 43.5, 48.1, 27.2).
template <int DT, int PER, bool TAIL>
__global__ __launch_bounds__(kPackThreads) void quant_short_kernel(QuantParams a)
{
    typedef typename Elem<DT>::store_t T;
    typedef typename Pack16<DT>::vec_t vec_t;
    constexpr int V = 8 / Elem<DT>::kPer16;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t row = (int64_t)blockIdx.x * (kPackThreads / kWave) + threadIdx.x / kWave;
    if (row >= a.rows)
        return;
    const T *src = static_cast<const T *>(a.X) + row * a.ldx;
    vec_t x[PER][V];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (i * kWave + lane) * 8 + v * Elem<DT>::kPer16;
            x[i][v] = vec_t{};
            if (col < a.K)
                x[i][v] = TAIL ? load16<DT>(src, col, a.K)
                               : *reinterpret_cast<const vec_t *>(src + col);
        }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        m = max(m, raw_max_bits<DT>(x[i]));
    m = wave_max(m);
    const float inv = row_inverse(m);
    if (lane == 0)
        a.scales[row] = row_scale(m);
    char *q = a.Q + row * a.Kq;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = (i * kWave + lane) * 8;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f[k] = Elem<DT>::widen(x[i][k / Elem<DT>::kPer16][k % Elem<DT>::kPer16]);
        if (col < a.Kq)
            put_codes(q, col, f, m, inv);
    }
}

// Longer rows: a workgroup per row.  Its values stay in registers between the
// maximum and the codes up to 8192 columns; the columns past that are read again.
// Eight waves a SIMD: left alone the compiler takes 114 registers for four (32768 rows of
// 4096 bf16 130 us, so 89; 4096 rows 20.1 and 16.6; a wave a row 85 and 19.8, but one row
// 4.2 for 2.5).
template <int DT>
__global__ __launch_bounds__(kPackThreads, 8) void quant_long_kernel(QuantParams a)
{
    typedef typename Elem<DT>::store_t T;
    constexpr int PER = 4, THREADS = kPackThreads;
    __shared__ uint32_t s_max[THREADS / kWave];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    char *q = a.Q + row * a.Kq;
    float f[PER][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = (i * THREADS + tid) * 8;
        if (col < a.K) {
            load8f<DT>(x, col, a.K, f[i]);
            m = max(m, abs_max_bits(f[i]));
        }
    }
    for (int col = (PER * THREADS + tid) * 8; col < a.K; col += THREADS * 8) {
        float g[8];
        load8f<DT>(x, col, a.K, g);
        m = max(m, abs_max_bits(g));
    }
    m = wave_max(m);
    if (tid % kWave == 0)
        s_max[tid / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w)
        m = max(m, s_max[w]);
    const float inv = row_inverse(m);
    if (tid == 0)
        a.scales[row] = row_scale(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int col = (i * THREADS + tid) * 8;
        if (col < a.K)
            put_codes(q, col, f[i], m, inv);
        else if (col < a.Kq)
            *reinterpret_cast<uint2 *>(q + col) = uint2{0, 0};
    }
    for (int col = (PER * THREADS + tid) * 8; col < a.Kq; col += THREADS * 8) {
        float g[8] = {};
        if (col < a.K)
            load8f<DT>(x, col, a.K, g);
        put_codes(q, col, g, m, inv);
    }
}

// Four lanes per block of 32, 8 columns each: a block's maximum takes two register
// moves, a lane 16 bytes of bf16 and stores 8 codes.  Bound by memory: 16384 rows of
// 4096 bf16 in 33 to 39 us (5.2 to 6.2 TB/s); back 31 us (6.5 TB/s, in part from cache).
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

// Packed rows as the bf16 rows that dW's reduction reads: 8192 rows of 2048 in 12 us
// (51 MB).  One workgroup per row at a time; as the copy in front of dW, an entry of
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

// A row of odd length starts at any 2-byte address, and the products' copies to LDS
// take aligned 16-byte pieces alone: such operands are copied once in front of them,
// zeros behind each row's end.  9 weights of 1034 rows of 1003 and 1001 rows of X
// (41 MB both ways): 11 us, a launch for each operand 15.
__global__ __launch_bounds__(kPackThreads) void pad_rows_kernel(PadParams a)
{
    for (int o = 0; o < a.num; ++o) {
        const PadOperand &p = a.op[o];
        const uint32_t cpr = (uint32_t)((p.cols + 7) / 8);
        const int64_t total = p.rows * cpr;
        for (int64_t base = (int64_t)blockIdx.x * kPackThreads; base < total;
             base += (int64_t)gridDim.x * kPackThreads) {
            const int64_t r0 = base / cpr;
            const uint32_t in = (uint32_t)(base - r0 * cpr) + threadIdx.x;
            const int64_t row = r0 + in / cpr;
            const int c = (int)(in % cpr);
            if (row >= p.rows)
                continue;
            if (p.m_sizes) {
                int64_t g = r0 / p.group_rows;  // uniform; a few rows may pass its end
                while (row >= (g + 1) * p.group_rows)
                    ++g;
                if (p.m_sizes[g] <= 0)
                    continue;
            }
            *reinterpret_cast<uint4 *>(p.dst + (row * cpr + c) * 16) = __builtin_bit_cast(
                uint4, load16<kBf16>(reinterpret_cast<const uint16_t *>(p.src) + row * p.cols,
                                     c * 8, p.cols));
        }
    }
}

namespace {

unsigned pack_grid(int64_t items)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(items, 256 * 32));
}

template <int DT, int PER>
void quant_short(const QuantParams &p, hipStream_t stream)
{
    constexpr int kRows = kPackThreads / kWave;
    const dim3 grid((unsigned)((p.rows + kRows - 1) / kRows)), block(kPackThreads);
    if (p.K % 8)
        hipLaunchKernelGGL((quant_short_kernel<DT, PER, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((quant_short_kernel<DT, PER, false>), grid, block, 0, stream, p);
}

template <int DT>
void quant_cfg(const QuantParams &p, hipStream_t stream)
{
    if (p.K <= kWave * 8)
        quant_short<DT, 1>(p, stream);
    else if (p.K <= kWave * 16)
        quant_short<DT, 2>(p, stream);
    else if (p.K <= kWave * 32)
        quant_short<DT, 4>(p, stream);
    else
        hipLaunchKernelGGL(quant_long_kernel<DT>, dim3((unsigned)p.rows), dim3(kPackThreads), 0,
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

hipError_t pad_rows_launch(const PadParams &p, hipStream_t stream)
{
    int64_t items = 1;
    for (int o = 0; o < p.num; ++o)
        items = std::max(items, (p.op[o].rows * ((p.op[o].cols + 7) / 8) + kPackThreads - 1) /
                                    kPackThreads);
    hipLaunchKernelGGL(pad_rows_kernel, dim3(pack_grid(items)), dim3(kPackThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace moegg
