// Kernel parameter blocks and host launchers of the feed-forward block: 8-bit
// integer products, the gated block and its backward pass, packed activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moegg.h"

namespace moegg {

// Columns of a packed block, and a row's columns in whole blocks.
constexpr int kPackBlock = 32;
__host__ __device__ inline int64_t packed_cols(int64_t cols)
{
    return (cols + kPackBlock - 1) / kPackBlock * kPackBlock;
}

// Y = grouped X W_e^T by 8-bit integers, or the gated block by bf16.  Rows of X
// and W are ldx and ldw bytes apart and hold K 16-bit units of reduction (two
// int8 each for the integers), K a multiple of 8.
struct BlockFwdParams {
    const char *X;
    const char *W;
    const float *x_scales;  // integers: [rows of X]
    const float *w_scales;  // integers: [E, N]
    const int32_t *m_sizes;
    const int32_t *gather;
    const float *topk_w;
    char *Y;          // [S, N], or H [S, N / 2] when gated
    char *A;          // gated: bf16 [S, N] or null
    char *Aq;         // gated: codes [S, 2 packed_cols(N / 2)] or null
    uint8_t *As;      //        and their exponents
    int32_t *err;
    int64_t S;
    int64_t ldx, ldw;
    int topk, E, N, K;
    uint32_t flags;
};

// dH = grouped dY W_e, and the gated activation's backward behind it.
struct GatedBwdParams {
    const char *dY;   // bf16, N columns, ldy bytes apart
    const char *W;    // bf16 [E, N, I], rows ldw bytes apart
    const int32_t *m_sizes;
    const int32_t *gather;
    const char *A;
    const char *Aq;
    const uint8_t *As;
    char *dA;         // [S, 2 I]
    char *H;          // [S, I] or null
    int32_t *err;
    int64_t S;
    int64_t ldy, ldw;
    int topk, E, N, I;
    uint32_t flags;
};

struct QuantParams {
    const void *X;
    int64_t ldx;
    char *Q;
    float *scales;
    int64_t rows;
    int K, Kq;
};

struct PackParams {
    const void *X;
    void *out;        // unpack: the values
    int64_t ldx;
    char *Q;
    uint8_t *S;
    int64_t rows;
    int cols;
};

// Packed rows expanded to bf16: out[p] = X[src(p)], src(p) = gather[p] / topk
// under PERMUTE_X for the positions below the sum of m_sizes (gather null: p).
struct UnpackRowsParams {
    const char *Q;
    const uint8_t *S;
    const int32_t *m_sizes;
    const int32_t *gather;
    char *out;
    int32_t *err;
    int64_t rows;
    int topk, E, cols;
};

// Rows of bf16 copied to rows of whole 16-byte chunks, for up to two operands in one
// launch: `rows` rows of `cols` columns, in groups of `group_rows`; a group whose
// entry of m_sizes is not positive is left out (m_sizes null: none).
struct PadOperand {
    const char *src;
    char *dst;
    const int32_t *m_sizes;
    int64_t rows, group_rows;
    int cols;
};
struct PadParams {
    PadOperand op[2];
    int num;
};
inline int64_t padded_row_bytes(int64_t cols)
{
    return (cols + 7) / 8 * 16;
}

// Whether rows of one expert are so few that vectors beat tiles, and that launch.
bool block_vec_pays(const BlockFwdParams &p, int cus);
hipError_t block_vec_launch(const BlockFwdParams &p, int cus, hipStream_t stream);
hipError_t i8_launch(const BlockFwdParams &p, int cus, hipStream_t stream);
// The two activations, compiled apart.
void gated_fwd_silu(const BlockFwdParams &p, int cus, hipStream_t stream);
void gated_fwd_gelu(const BlockFwdParams &p, int cus, hipStream_t stream);
inline hipError_t gated_fwd_launch(const BlockFwdParams &p, int cus, hipStream_t stream)
{
    if (!p.A && !p.Aq && block_vec_pays(p, cus))
        return block_vec_launch(p, cus, stream);
    if (p.flags & MOEGG_GATED_GELU)
        gated_fwd_gelu(p, cus, stream);
    else
        gated_fwd_silu(p, cus, stream);
    return hipGetLastError();
}
hipError_t gated_bwd_launch(const GatedBwdParams &p, int cus, hipStream_t stream);
hipError_t quant_rows_launch(const QuantParams &p, int dtype, hipStream_t stream);
hipError_t pack8_launch(const PackParams &p, int dtype, hipStream_t stream);
hipError_t unpack8_launch(const PackParams &p, int dtype, hipStream_t stream);
hipError_t unpack_rows_launch(const UnpackRowsParams &p, int cus, hipStream_t stream);
hipError_t pad_rows_launch(const PadParams &p, hipStream_t stream);

}  // namespace moegg
