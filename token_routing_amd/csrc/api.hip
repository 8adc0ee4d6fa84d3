// extern "C" entry points of libmoegg.so: argument checks, then launches.
//
// The checks are the preconditions the pages' launchers assert
// (grouped_gemm_forward, grouped_gemm_dX, grouped_gemm_dW and
// check_valid_config_* in unsloth grouped_gemm/interface.py;
// _allocate_asymmetric_dual_outputs in wall_x/fusions/backend.py), turned into
// status codes.  Every check runs on the host before anything is enqueued, so
// a rejected call touches neither the device nor the stream.
#include "common.h"

#include "../../include/moegg.h"

#include "gemm_params.h"
#include "layer_params.h"
#include "lora_params.h"

namespace {

constexpr int kMaxDevices = 64;
int g_cus[kMaxDevices];

// Compute units of the current device (queried once per device).
int device_cus(int *cus)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return -1;
    if (g_cus[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n < 1)
            return -1;
        g_cus[dev] = n;
    }
    *cus = g_cus[dev];
    return 0;
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// bf16 (fp32) elements need 2- (4-) byte alignment on every path.
bool aligned2(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 1u) == 0;
}
bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

// A launch has fewer than 2^32 threads.
constexpr int64_t kMaxThreads = (int64_t)1 << 32;

bool known_dtype(int32_t dtype)
{
    return dtype == MOEGG_BF16 || dtype == MOEGG_FP16 || dtype == MOEGG_FP32;
}
bool aligned_elem(const void *p, int32_t dtype)
{
    return dtype == MOEGG_FP32 ? aligned4(p) : aligned2(p);
}

// The tiled kernels move rows as 16-byte chunks: row lengths that are
// multiples of 8 elements and 16-byte aligned operands.  Other shapes take
// the any-shape launches.
bool tiled_rows(int64_t n, int64_t k)
{
    return n % 8 == 0 && k % 8 == 0;
}

moegg_status check_gemm_common(int32_t num_tokens, int32_t topk, int32_t E, int32_t N, int32_t K)
{
    if (num_tokens < 0 || topk < 1 || E < 1 || E > MOEGG_MAX_EXPERTS || N < 1 || K < 1)
        return MOEGG_ESHAPE;
    if ((int64_t)num_tokens * topk > INT32_MAX)
        return MOEGG_ESHAPE;
    return MOEGG_OK;
}

// Gather indices are required with a permute flag whenever there are rows.
moegg_status check_permute_flags(uint32_t flags, const int32_t *gather_idx, int64_t S)
{
    const bool px = flags & MOEGG_PERMUTE_X, py = flags & MOEGG_PERMUTE_Y;
    if (px && py)
        return MOEGG_EINVAL;  // the pages' launcher rejects both permutes at once
    if ((px || py) && S > 0 && gather_idx == nullptr)
        return MOEGG_EINVAL;  // gather_indices required with a permute flag
    return MOEGG_OK;
}

// Operands are addressed through buffer resources with 32-bit offsets and an
// out-of-range sentinel at 2^31: every operand must stay below 2 GiB.
constexpr int64_t kMaxOperandBytes = (int64_t)1 << 31;

bool fits(int64_t rows, int64_t row_elems, int64_t elem_bytes = 2)
{
    return rows * row_elems * elem_bytes < kMaxOperandBytes;
}

moegg_status from_hip(hipError_t e)
{
    return e == hipSuccess ? MOEGG_OK : MOEGG_EHIP;
}

}  // namespace

extern "C" {

const char *moegg_status_string(moegg_status s)
{
    switch (s) {
    case MOEGG_OK: return "ok";
    case MOEGG_EINVAL: return "invalid argument or flag combination";
    case MOEGG_ESHAPE: return "invalid or inconsistent sizes";
    case MOEGG_EUNSUPPORTED: return "unsupported option";
    case MOEGG_EWORKSPACE: return "workspace missing or too small";
    case MOEGG_EHIP: return "HIP error";
    }
    return "unknown status";
}

int32_t moegg_version(void)
{
    return 102;
}

size_t moegg_route_workspace_bytes(int64_t num_slots, int32_t num_experts)
{
    if (num_slots <= 0 || num_experts < 1)
        return 0;
    return (size_t)moegg::route_chunks(num_slots) * (size_t)num_experts * sizeof(int32_t);
}

moegg_status moegg_route(const int32_t *topk_ids, int32_t num_tokens, int32_t topk,
                         int32_t num_experts, int32_t block_m, int32_t *m_sizes,
                         int32_t *offsets, int32_t *padded_offsets, int32_t *tile_offsets,
                         int32_t *gather_idx, int32_t *scatter_idx, void *workspace,
                         size_t workspace_bytes, int32_t *error_flags, void *stream)
{
    if (num_tokens < 0 || topk < 1 || num_experts < 1 || num_experts > MOEGG_MAX_EXPERTS ||
        block_m < 1)
        return MOEGG_ESHAPE;
    const int64_t S = (int64_t)num_tokens * topk;
    if (S > INT32_MAX)
        return MOEGG_ESHAPE;
    if (m_sizes == nullptr || offsets == nullptr)
        return MOEGG_EINVAL;
    if (S > 0 && (topk_ids == nullptr || gather_idx == nullptr))
        return MOEGG_EINVAL;
    const size_t need = moegg_route_workspace_bytes(S, num_experts);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return MOEGG_EWORKSPACE;
    return from_hip(moegg::route_launch(topk_ids, S, num_experts, block_m, m_sizes, offsets,
                                        padded_offsets, tile_offsets, gather_idx, scatter_idx,
                                        static_cast<int32_t *>(workspace), error_flags,
                                        static_cast<hipStream_t>(stream)));
}

moegg_status moegg_route_noalloc(const int32_t *topk_ids, int32_t num_tokens, int32_t topk,
                                 int32_t num_experts, int32_t block_m, int32_t *m_sizes,
                                 int32_t *offsets, int32_t *padded_offsets, int32_t *tile_offsets,
                                 int32_t *gather_idx, int32_t *scatter_idx, int32_t *error_flags,
                                 void *stream)
{
    if (num_tokens < 0 || topk < 1 || num_experts < 1 || num_experts > MOEGG_MAX_EXPERTS ||
        block_m < 1)
        return MOEGG_ESHAPE;
    const int64_t S = (int64_t)num_tokens * topk;
    if (S > INT32_MAX)
        return MOEGG_ESHAPE;
    if (m_sizes == nullptr || offsets == nullptr)
        return MOEGG_EINVAL;
    if (S > 0 && (topk_ids == nullptr || gather_idx == nullptr))
        return MOEGG_EINVAL;
    if (moegg_route_workspace_bytes(S, num_experts) > MOEGG_ROUTE_NOALLOC_MAX_BYTES)
        return MOEGG_EWORKSPACE;  // more per-chunk counts than the static array holds
    int32_t *counts = nullptr;
    hipError_t e = moegg::route_scratch(&counts);
    if (e != hipSuccess)
        return MOEGG_EHIP;
    return from_hip(moegg::route_launch(topk_ids, S, num_experts, block_m, m_sizes, offsets,
                                        padded_offsets, tile_offsets, gather_idx, scatter_idx,
                                        counts, error_flags, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_grouped_gemm_fwd(const void *X, const void *W, const int32_t *m_sizes,
                                    const int32_t *gather_idx, const float *topk_weights,
                                    int32_t num_tokens, int32_t topk, int32_t num_experts,
                                    int32_t N, int32_t K, uint32_t flags, void *Y,
                                    int32_t *error_flags, void *stream)
{
    moegg_status st = check_gemm_common(num_tokens, topk, num_experts, N, K);
    if (st != MOEGG_OK)
        return st;
    if (flags & ~(MOEGG_PERMUTE_X | MOEGG_PERMUTE_Y | MOEGG_FUSE_MUL_POST | MOEGG_GATED_SILU))
        return MOEGG_EINVAL;
    if ((st = check_permute_flags(flags, gather_idx, (int64_t)num_tokens * topk)) != MOEGG_OK)
        return st;
    if ((flags & MOEGG_FUSE_MUL_POST) && !(flags & MOEGG_PERMUTE_Y))
        return MOEGG_EINVAL;  // the gate multiply is fused only with permute_y
    if ((flags & MOEGG_GATED_SILU) && (flags & (MOEGG_PERMUTE_Y | MOEGG_FUSE_MUL_POST)))
        return MOEGG_EINVAL;  // the activation belongs to the first GEMM
    if ((flags & MOEGG_GATED_SILU) && N % 2 != 0)
        return MOEGG_ESHAPE;  // W rows come in (gate, linear) pairs
    if ((flags & MOEGG_FUSE_MUL_POST) && num_tokens > 0 && topk_weights == nullptr)
        return MOEGG_EINVAL;
    if (num_tokens == 0)
        return MOEGG_OK;
    if (X == nullptr || W == nullptr || m_sizes == nullptr || Y == nullptr)
        return MOEGG_EINVAL;
    if (!aligned2(X) || !aligned2(W) || !aligned2(Y))
        return MOEGG_ESHAPE;
    const bool tiled = tiled_rows(N, K) && (!(flags & MOEGG_GATED_SILU) || N % 16 == 0) &&
                       aligned16(X) && aligned16(W) && aligned16(Y);
    {
        const int64_t S = (int64_t)num_tokens * topk;
        const int64_t x_rows = (flags & MOEGG_PERMUTE_X) ? num_tokens : S;
        if (!fits(x_rows, K) || !fits(N, K))
            return MOEGG_ESHAPE;
    }
    int cus = 0;
    if (device_cus(&cus) != 0)
        return MOEGG_EHIP;
    moegg::FwdParams p;
    p.X = static_cast<const char *>(X);
    p.W = static_cast<const char *>(W);
    p.m_sizes = m_sizes;
    p.gather = gather_idx;
    p.topk_w = topk_weights;
    p.Y = static_cast<char *>(Y);
    p.err = error_flags;
    p.S = (int64_t)num_tokens * topk;
    p.topk = topk;
    p.E = num_experts;
    p.N = N;
    p.K = K;
    p.flags = flags;
    return from_hip(tiled ? moegg::fwd_launch(p, cus, static_cast<hipStream_t>(stream))
                          : moegg::fwd_any_launch(p, cus, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_grouped_gemm_dX(const void *dY, const void *W, const int32_t *m_sizes,
                                   const int32_t *gather_idx, int32_t num_tokens, int32_t topk,
                                   int32_t num_experts, int32_t N, int32_t K, uint32_t flags,
                                   void *dX, void *workspace, size_t workspace_bytes,
                                   int32_t *error_flags, void *stream)
{
    moegg_status st = check_gemm_common(num_tokens, topk, num_experts, N, K);
    if (st != MOEGG_OK)
        return st;
    if (flags & MOEGG_FUSE_MUL_POST)
        return MOEGG_EUNSUPPORTED;  // fuse_mul is for inference only
    if (flags & ~(MOEGG_PERMUTE_X | MOEGG_PERMUTE_Y))
        return MOEGG_EINVAL;
    if ((st = check_permute_flags(flags, gather_idx, (int64_t)num_tokens * topk)) != MOEGG_OK)
        return st;
    if (num_tokens == 0)
        return MOEGG_OK;
    if (dY == nullptr || W == nullptr || m_sizes == nullptr || dX == nullptr)
        return MOEGG_EINVAL;
    if (!aligned2(dY) || !aligned2(W) || !aligned2(dX) || !aligned16(workspace))
        return MOEGG_ESHAPE;
    if (!fits((int64_t)num_tokens * topk, N) || !fits(N, K))
        return MOEGG_ESHAPE;
    const bool tiled = tiled_rows(N, K) && aligned16(dY) && aligned16(W) && aligned16(dX);
    int cus = 0;
    if (device_cus(&cus) != 0)
        return MOEGG_EHIP;
    const int64_t ws_need =
        tiled ? moegg::dx_workspace_bytes((int64_t)num_tokens * topk, num_experts, N, K, cus) : 0;
    if (workspace != nullptr && (int64_t)workspace_bytes < ws_need)
        return MOEGG_EWORKSPACE;
    moegg::DxParams p;
    p.ws = workspace != nullptr && ws_need > 0 ? static_cast<char *>(workspace) : nullptr;
    p.dY = static_cast<const char *>(dY);
    p.W = static_cast<const char *>(W);
    p.m_sizes = m_sizes;
    p.gather = gather_idx;
    p.dX = static_cast<char *>(dX);
    p.err = error_flags;
    p.S = (int64_t)num_tokens * topk;
    p.topk = topk;
    p.E = num_experts;
    p.N = N;
    p.K = K;
    p.flags = flags;
    return from_hip(tiled ? moegg::dx_launch(p, cus, static_cast<hipStream_t>(stream))
                          : moegg::dx_any_launch(p, cus, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_grouped_gemm_dW(const void *X, const void *dY, const int32_t *m_sizes,
                                   const int32_t *gather_idx, int32_t num_tokens, int32_t topk,
                                   int32_t num_experts, int32_t N, int32_t K, uint32_t flags,
                                   void *dW, void *workspace, size_t workspace_bytes,
                                   int32_t *error_flags, void *stream)
{
    moegg_status st = check_gemm_common(num_tokens, topk, num_experts, N, K);
    if (st != MOEGG_OK)
        return st;
    if (flags & MOEGG_FUSE_MUL_POST)
        return MOEGG_EUNSUPPORTED;
    if (flags & ~(MOEGG_PERMUTE_X | MOEGG_PERMUTE_Y | MOEGG_DW_FP32_OUT))
        return MOEGG_EINVAL;
    if ((st = check_permute_flags(flags, gather_idx, (int64_t)num_tokens * topk)) != MOEGG_OK)
        return st;
    if (dW == nullptr || m_sizes == nullptr)
        return MOEGG_EINVAL;
    if (num_tokens > 0 && (X == nullptr || dY == nullptr))
        return MOEGG_EINVAL;
    if (!aligned2(X) || !aligned2(dY) || !aligned2(dW) || !aligned16(workspace))
        return MOEGG_ESHAPE;
    if ((flags & MOEGG_DW_FP32_OUT) && !aligned4(dW))
        return MOEGG_ESHAPE;
    {
        const int64_t S = (int64_t)num_tokens * topk;
        const int64_t x_rows = (flags & MOEGG_PERMUTE_X) ? num_tokens : S;
        if (!fits(x_rows, K) || !fits(S, N))
            return MOEGG_ESHAPE;
    }
    const bool tiled = tiled_rows(N, K) && aligned16(X) && aligned16(dY) && aligned16(dW);
    const int64_t ws_need =
        tiled ? moegg::dw_workspace_bytes((int64_t)num_tokens * topk, num_experts, N, K) : 0;
    const bool use_ws = workspace != nullptr && ws_need > 0;
    if (workspace != nullptr && (int64_t)workspace_bytes < ws_need)
        return MOEGG_EWORKSPACE;
    // Room for X's rows in expert order after the partials: gather them first.
    // The copy is an operand of the reduction like X itself, so it must stay
    // below 2 GiB too; a larger one keeps the gather inside the reduction.
    const int64_t xg_off = moegg::dw_gather_offset((int64_t)num_tokens * topk, num_experts, N, K);
    const int64_t xg_bytes = (int64_t)num_tokens * topk * K * 2;
    const bool use_xg = tiled && workspace != nullptr && (flags & MOEGG_PERMUTE_X) && xg_bytes > 0 &&
                        fits((int64_t)num_tokens * topk, K) &&
                        (int64_t)workspace_bytes >= xg_off + xg_bytes;
    int cus = 0;
    if (device_cus(&cus) != 0)
        return MOEGG_EHIP;
    // T = 0 still writes dW: every expert is empty, so dW is all zeros.
    moegg::DwParams p;
    p.X = static_cast<const char *>(X);
    p.dY = static_cast<const char *>(dY);
    p.m_sizes = m_sizes;
    p.gather = gather_idx;
    p.dW = static_cast<char *>(dW);
    p.err = error_flags;
    p.S = (int64_t)num_tokens * topk;
    p.topk = topk;
    p.E = num_experts;
    p.N = N;
    p.K = K;
    p.flags = flags;
    p.topk_div = moegg::make_fastdiv((uint32_t)topk);
    p.ws = use_ws ? static_cast<char *>(workspace) : nullptr;
    p.xg = use_xg ? static_cast<char *>(workspace) + xg_off : nullptr;
    p.split_rows = use_ws ? moegg::dw_split_rows(p.S, N, K) : 0;
    return from_hip(tiled ? moegg::dw_launch(p, cus, static_cast<hipStream_t>(stream))
                          : moegg::dw_any_launch(p, cus, static_cast<hipStream_t>(stream)));
}

size_t moegg_grouped_gemm_dX_workspace_bytes(int32_t num_tokens, int32_t topk,
                                             int32_t num_experts, int32_t N, int32_t K)
{
    if (check_gemm_common(num_tokens, topk, num_experts, N, K) != MOEGG_OK || !tiled_rows(N, K))
        return 0;
    int cus = 0;
    if (device_cus(&cus) != 0)
        return 0;
    return (size_t)moegg::dx_workspace_bytes((int64_t)num_tokens * topk, num_experts, N, K, cus);
}

size_t moegg_grouped_gemm_dW_workspace_bytes(int32_t num_tokens, int32_t topk,
                                             int32_t num_experts, int32_t N, int32_t K)
{
    if (check_gemm_common(num_tokens, topk, num_experts, N, K) != MOEGG_OK || !tiled_rows(N, K))
        return 0;
    return (size_t)moegg::dw_workspace_bytes((int64_t)num_tokens * topk, num_experts, N, K);
}

size_t moegg_grouped_gemm_dW_gather_workspace_bytes(int32_t num_tokens, int32_t topk,
                                                    int32_t num_experts, int32_t N, int32_t K)
{
    if (check_gemm_common(num_tokens, topk, num_experts, N, K) != MOEGG_OK || !tiled_rows(N, K))
        return 0;
    const int64_t S = (int64_t)num_tokens * topk;
    // No copy: the rows are gathered inside the reduction.
    if (!fits(S, K) || moegg::dw_short_launch(S, num_tokens, num_experts, N, K))
        return (size_t)moegg::dw_workspace_bytes(S, num_experts, N, K);
    return (size_t)(moegg::dw_gather_offset(S, num_experts, N, K) + S * K * 2);
}

moegg_status moegg_grouped_gemm_groups(const moegg_group *groups, int32_t num_groups,
                                       int32_t trans_b, void *stream)
{
    if (groups == nullptr || (trans_b != 0 && trans_b != 1))
        return MOEGG_EINVAL;
    if (num_groups < 1 || num_groups > MOEGG_MAX_GROUPS)
        return MOEGG_ESHAPE;
    moegg::GroupsParams p;
    p.num = num_groups;
    bool any = false, tiled = true;
    for (int i = 0; i < num_groups; ++i) {
        const moegg_group &g = groups[i];
        if (g.m < 0 || g.n < 1 || g.k < 1)
            return MOEGG_ESHAPE;
        if (g.ldx < g.k || g.ldy < g.n || g.ldw < (trans_b ? g.k : g.n))
            return MOEGG_ESHAPE;
        if (g.m > 0 && (g.x == nullptr || g.w == nullptr || g.y == nullptr))
            return MOEGG_EINVAL;
        if (!aligned2(g.x) || !aligned2(g.w) || !aligned2(g.y))
            return MOEGG_ESHAPE;
        tiled &= !(g.n % 8 || g.k % 8 || g.ldx % 8 || g.ldw % 8 || g.ldy % 8) &&
                 aligned16(g.x) && aligned16(g.w) && aligned16(g.y);
        if (!fits(g.m, g.ldx) || !fits(trans_b ? g.n : g.k, g.ldw))
            return MOEGG_ESHAPE;
        any |= g.m > 0;
        p.g[i] = g;
    }
    if (!any)
        return MOEGG_OK;
    int cus = 0;
    if (device_cus(&cus) != 0)
        return MOEGG_EHIP;
    return from_hip(tiled ? moegg::groups_launch(p, trans_b, cus, static_cast<hipStream_t>(stream))
                          : moegg::groups_any_launch(p, trans_b, cus,
                                                     static_cast<hipStream_t>(stream)));
}

// Shared checks of the combine entry points.
static moegg_status check_combine(int64_t num_tokens, int32_t topk, int32_t N, int64_t y_rows,
                                  const int32_t *scatter)
{
    if (num_tokens < 0 || topk < 1 || N < 1 || y_rows < 0)
        return MOEGG_ESHAPE;
    if (num_tokens * topk > INT32_MAX)
        return MOEGG_ESHAPE;
    if (scatter == nullptr && y_rows < num_tokens * topk)
        return MOEGG_ESHAPE;  // slot-order Y has one row per slot
    if (y_rows * (int64_t)N * 2 >= ((int64_t)1 << 40) || num_tokens * (int64_t)N * 4 >= ((int64_t)1 << 40))
        return MOEGG_ESHAPE;
    return MOEGG_OK;
}

moegg_status moegg_combine(const void *Y, const int32_t *scatter_idx, const float *topk_weights,
                           int64_t num_tokens, int32_t topk, int32_t N, int64_t y_rows,
                           uint32_t flags, void *out, int32_t *error_flags, void *stream)
{
    moegg_status st = check_combine(num_tokens, topk, N, y_rows, scatter_idx);
    if (st != MOEGG_OK)
        return st;
    if (flags & ~(uint32_t)MOEGG_COMBINE_FP32_OUT)
        return MOEGG_EINVAL;
    if (num_tokens == 0)
        return MOEGG_OK;
    if (!Y || !out || !aligned2(Y) || !aligned2(out))
        return MOEGG_EINVAL;
    if ((flags & MOEGG_COMBINE_FP32_OUT) && !aligned4(out))
        return MOEGG_EINVAL;
    const bool tiled = N % 8 == 0 && aligned16(Y) && aligned16(out);
    moegg::CombineParams p;
    p.Y = static_cast<const char *>(Y);
    p.scatter = scatter_idx;
    p.weights = topk_weights;
    p.out = static_cast<char *>(out);
    p.err = error_flags;
    p.T = num_tokens;
    p.y_rows = y_rows;
    p.topk = topk;
    p.N = N;
    p.f32_out = flags & MOEGG_COMBINE_FP32_OUT;
    return from_hip(tiled ? moegg::combine_launch(p, static_cast<hipStream_t>(stream))
                          : moegg::combine_any_launch(p, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_combine_bwd(const void *dOut, const void *Y, const int32_t *scatter_idx,
                               const float *topk_weights, int64_t num_tokens, int32_t topk,
                               int32_t N, int64_t y_rows, void *dY, float *dw,
                               int32_t *error_flags, void *stream)
{
    moegg_status st = check_combine(num_tokens, topk, N, y_rows, scatter_idx);
    if (st != MOEGG_OK)
        return st;
    if (num_tokens == 0)
        return MOEGG_OK;
    if (!dOut || !dY || !aligned2(dOut) || !aligned2(dY))
        return MOEGG_EINVAL;
    if (dw && (!Y || !aligned2(Y)))
        return MOEGG_EINVAL;  // the weight gradient reads the forward input
    const bool tiled = N % 8 == 0 && aligned16(dOut) && aligned16(dY) && (!dw || aligned16(Y));
    moegg::CombineBwdParams p;
    p.dOut = static_cast<const char *>(dOut);
    p.Y = static_cast<const char *>(Y);
    p.scatter = scatter_idx;
    p.weights = topk_weights;
    p.dY = static_cast<char *>(dY);
    p.dw = dw;
    p.err = error_flags;
    p.T = num_tokens;
    p.y_rows = y_rows;
    p.topk = topk;
    p.N = N;
    return from_hip(tiled ? moegg::combine_bwd_launch(p, static_cast<hipStream_t>(stream))
                          : moegg::combine_bwd_any_launch(p, static_cast<hipStream_t>(stream)));
}

// Whether a [T, E] output of the gate overlaps its logits other than element
// for element (in place).
static bool beside_logits(const void *out, int64_t out_size, const void *logits, int32_t dtype,
                          int64_t ld, int64_t T, int64_t E)
{
    const int64_t size = dtype == MOEGG_FP32 ? 4 : 2;
    const int64_t po = reinterpret_cast<intptr_t>(out), pl = reinterpret_cast<intptr_t>(logits);
    if (!out || po >= pl + ((T - 1) * ld + E) * size || pl >= po + T * E * out_size)
        return false;
    return po != pl || out_size != size || (ld != E && T > 1);
}

// Shared checks of the gate entry points.
static moegg_status check_gate(const void *logits, int32_t dtype, int64_t ld, int64_t num_tokens,
                               int32_t E, int32_t topk, float scale, uint32_t flags)
{
    if (num_tokens < 0 || E < 1 || E > MOEGG_MAX_EXPERTS || topk < 1 || topk > E ||
        topk > MOEGG_MAX_TOPK || ld < E)
        return MOEGG_ESHAPE;
    if (num_tokens > INT32_MAX / topk || num_tokens >= kMaxThreads / 64 ||
        ld > ((int64_t)1 << 40) / (num_tokens + 1) / 4)
        return MOEGG_ESHAPE;
    if (!known_dtype(dtype) || (flags & ~(uint32_t)(MOEGG_GATE_SIGMOID | MOEGG_GATE_RENORM)) ||
        !(scale - scale == 0.0f))
        return MOEGG_EINVAL;
    if (num_tokens > 0 && (!logits || !aligned_elem(logits, dtype)))
        return MOEGG_EINVAL;
    return MOEGG_OK;
}

moegg_status moegg_gate(const void *logits, int32_t dtype, int64_t ld_logits, const float *bias,
                        int64_t num_tokens, int32_t num_experts, int32_t topk, int32_t n_groups,
                        int32_t topk_groups, float scale, uint32_t flags, int32_t *topk_ids,
                        float *topk_weights, float *scores, int32_t *error_flags, void *stream)
{
    moegg_status st =
        check_gate(logits, dtype, ld_logits, num_tokens, num_experts, topk, scale, flags);
    if (st != MOEGG_OK)
        return st;
    if (n_groups < 1 || n_groups > MOEGG_MAX_GATE_GROUPS || num_experts % n_groups != 0 ||
        topk_groups < 1 || topk_groups > n_groups || topk > topk_groups * (num_experts / n_groups))
        return MOEGG_ESHAPE;
    if (num_tokens == 0)
        return MOEGG_OK;
    if (!topk_ids || !topk_weights || !aligned4(topk_ids) || !aligned4(topk_weights) ||
        !aligned4(scores) || !aligned4(bias))
        return MOEGG_EINVAL;
    // With a bias or groups the picks' logits are read again after scores are written.
    if (beside_logits(scores, 4, logits, dtype, ld_logits, num_tokens, num_experts) ||
        (scores == logits && (bias || n_groups > 1)))
        return MOEGG_EINVAL;
    moegg::GateParams p;
    p.logits = logits;
    p.bias = bias;
    p.ids = topk_ids;
    p.weights = topk_weights;
    p.scores = scores;
    p.err = error_flags;
    p.T = num_tokens;
    p.ld = ld_logits;
    p.E = num_experts;
    p.topk = topk;
    p.n_groups = n_groups;
    p.topk_groups = topk_groups;
    p.dtype = dtype;
    p.scale = scale;
    p.sigmoid = flags & MOEGG_GATE_SIGMOID;
    p.renorm = flags & MOEGG_GATE_RENORM;
    return from_hip(moegg::gate_launch(p, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_gate_bwd(const void *logits, int32_t dtype, int64_t ld_logits,
                            const int32_t *topk_ids, const float *dweights, const float *dscores,
                            int64_t num_tokens, int32_t num_experts, int32_t topk, float scale,
                            uint32_t flags, void *dlogits, int32_t *error_flags, void *stream)
{
    moegg_status st =
        check_gate(logits, dtype, ld_logits, num_tokens, num_experts, topk, scale, flags);
    if (st != MOEGG_OK)
        return st;
    if (num_tokens == 0)
        return MOEGG_OK;
    if (!topk_ids || !dweights || !dlogits || !aligned4(topk_ids) || !aligned4(dweights) ||
        !aligned4(dscores) || !aligned_elem(dlogits, dtype))
        return MOEGG_EINVAL;
    if (beside_logits(dlogits, dtype == MOEGG_FP32 ? 4 : 2, logits, dtype, ld_logits, num_tokens,
                      num_experts))
        return MOEGG_EINVAL;
    moegg::GateBwdParams p;
    p.logits = logits;
    p.ids = topk_ids;
    p.dweights = dweights;
    p.dscores = dscores;
    p.dlogits = dlogits;
    p.err = error_flags;
    p.T = num_tokens;
    p.ld = ld_logits;
    p.E = num_experts;
    p.topk = topk;
    p.dtype = dtype;
    p.scale = scale;
    p.sigmoid = flags & MOEGG_GATE_SIGMOID;
    p.renorm = flags & MOEGG_GATE_RENORM;
    return from_hip(moegg::gate_bwd_launch(p, static_cast<hipStream_t>(stream)));
}

// Shared checks of the permute and unpermute entry points: tok holds [T, K]
// rows, sorted the [rows, K] ones.
static moegg_status check_sort(const void *tok, const void *sorted, int32_t dtype,
                               const int32_t *map, const float *weights, int64_t num_tokens,
                               int32_t topk, int32_t K, int64_t rows)
{
    constexpr int64_t kMax = (int64_t)1 << 38;  // elements: 2^40 bytes of fp32
    if (num_tokens < 0 || topk < 1 || K < 1 || K > (1 << 30) || rows < 0 || rows > INT32_MAX)
        return MOEGG_ESHAPE;
    // a workgroup of 256 threads a token, and up to 1088 for pad rows
    if (num_tokens > INT32_MAX / topk || num_tokens >= kMaxThreads / 256 - 2048 ||
        num_tokens > kMax / K || rows > kMax / K)
        return MOEGG_ESHAPE;
    if (!known_dtype(dtype))
        return MOEGG_EINVAL;
    if (num_tokens > 0 && (!tok || !map || !aligned_elem(tok, dtype) || !aligned4(map) ||
                           !aligned4(weights)))
        return MOEGG_EINVAL;
    if (rows > 0 && num_tokens > 0 && (!sorted || !aligned_elem(sorted, dtype)))
        return MOEGG_EINVAL;
    return MOEGG_OK;
}

// Whether two matrices of [rows, K] elements share memory; of one place and
// size they may where that is said (the kernels then read an element before
// they write it).
static bool sort_overlap(const void *a, int64_t rows_a, const void *b, int64_t rows_b, int32_t K,
                         int32_t dtype, bool in_place)
{
    const int64_t row = (int64_t)K * (dtype == MOEGG_FP32 ? 4 : 2);
    const int64_t pa = reinterpret_cast<intptr_t>(a), pb = reinterpret_cast<intptr_t>(b);
    return a && b && rows_a > 0 && rows_b > 0 && pa < pb + rows_b * row &&
           pb < pa + rows_a * row && !(in_place && pa == pb);
}

// The padded layout's metadata: both offset arrays or neither.
static moegg_status check_padded(const int32_t *offsets, const int32_t *padded, int32_t E,
                                 const void *sorted, int32_t dtype, int64_t rows)
{
    if (!offsets != !padded)
        return MOEGG_EINVAL;
    if (!padded)
        return MOEGG_OK;
    if (E < 1 || E > MOEGG_MAX_EXPERTS)
        return MOEGG_ESHAPE;
    if (!aligned4(offsets) || !aligned4(padded))
        return MOEGG_EINVAL;
    if (rows > 0 && (!sorted || !aligned_elem(sorted, dtype)))
        return MOEGG_EINVAL;
    return MOEGG_OK;
}

moegg_status moegg_permute(const void *X, int32_t dtype, const int32_t *scatter_idx,
                           const float *topk_weights, const int32_t *offsets,
                           const int32_t *padded_offsets, int64_t num_tokens, int32_t topk,
                           int32_t num_experts, int32_t K, int64_t rows, void *Xs,
                           int32_t *row_map, int32_t *error_flags, void *stream)
{
    moegg_status st =
        check_sort(X, Xs, dtype, scatter_idx, topk_weights, num_tokens, topk, K, rows);
    if (st == MOEGG_OK)
        st = check_padded(offsets, padded_offsets, num_experts, Xs, dtype, rows);
    if (st != MOEGG_OK)
        return st;
    if (num_tokens > 0 &&
        ((padded_offsets && (!row_map || row_map == scatter_idx)) || !aligned4(row_map)))
        return MOEGG_EINVAL;
    if (sort_overlap(Xs, rows, X, num_tokens, K, dtype, false))
        return MOEGG_EINVAL;
    moegg::SpreadParams p = {};
    p.src = X;
    p.map = scatter_idx;
    p.weights = topk_weights;
    p.offsets = offsets;
    p.padded = padded_offsets;
    p.dst = Xs;
    p.row_map = row_map;
    p.err = error_flags;
    p.T = num_tokens;
    p.rows = rows;
    p.topk = topk;
    p.E = num_experts;
    p.K = K;
    return from_hip(moegg::spread_launch(p, dtype, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_permute_bwd(const void *dXs, int32_t dtype, const void *X,
                               const int32_t *row_map, const float *topk_weights,
                               int64_t num_tokens, int32_t topk, int32_t K, int64_t rows, void *dX,
                               float *dw, int32_t *error_flags, void *stream)
{
    moegg_status st = check_sort(dX, dXs, dtype, row_map, topk_weights, num_tokens, topk, K, rows);
    if (st != MOEGG_OK || num_tokens == 0)
        return st;
    if (dw && (!X || !aligned_elem(X, dtype) || !aligned4(dw)))
        return MOEGG_EINVAL;
    if (sort_overlap(dX, num_tokens, dXs, rows, K, dtype, false) ||
        (dw && sort_overlap(dX, num_tokens, X, num_tokens, K, dtype, true)))
        return MOEGG_EINVAL;
    moegg::CollectParams p = {};
    p.rows_in = dXs;
    p.other = dw ? X : nullptr;
    p.map = row_map;
    p.weights = topk_weights;
    p.out = dX;
    p.dw = dw;
    p.err = error_flags;
    p.T = num_tokens;
    p.rows = rows;
    p.topk = topk;
    p.K = K;
    return from_hip(moegg::collect_launch(p, dtype, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_unpermute(const void *Y, int32_t dtype, const int32_t *row_map,
                             const float *topk_weights, const void *base, int64_t num_tokens,
                             int32_t topk, int32_t K, int64_t rows, void *out,
                             int32_t *error_flags, void *stream)
{
    moegg_status st = check_sort(out, Y, dtype, row_map, topk_weights, num_tokens, topk, K, rows);
    if (st != MOEGG_OK || num_tokens == 0)
        return st;
    if (base && !aligned_elem(base, dtype))
        return MOEGG_EINVAL;
    if (sort_overlap(out, num_tokens, Y, rows, K, dtype, false) ||
        sort_overlap(out, num_tokens, base, num_tokens, K, dtype, true))
        return MOEGG_EINVAL;
    moegg::CollectParams p = {};
    p.rows_in = Y;
    p.base = base;
    p.map = row_map;
    p.weights = topk_weights;
    p.out = out;
    p.err = error_flags;
    p.T = num_tokens;
    p.rows = rows;
    p.topk = topk;
    p.K = K;
    return from_hip(moegg::collect_launch(p, dtype, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_unpermute_bwd(const void *dOut, int32_t dtype, const void *Y,
                                 const int32_t *row_map, const float *topk_weights,
                                 const int32_t *offsets, const int32_t *padded_offsets,
                                 int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t K,
                                 int64_t rows, void *dY, float *dw, int32_t *error_flags,
                                 void *stream)
{
    moegg_status st =
        check_sort(dOut, dY, dtype, row_map, topk_weights, num_tokens, topk, K, rows);
    if (st == MOEGG_OK)
        st = check_padded(offsets, padded_offsets, num_experts, dY, dtype, rows);
    if (st != MOEGG_OK)
        return st;
    if (num_tokens > 0 && dw && ((rows > 0 && !Y) || !aligned_elem(Y, dtype) || !aligned4(dw)))
        return MOEGG_EINVAL;
    if (sort_overlap(dY, rows, dOut, num_tokens, K, dtype, false) ||
        (dw && sort_overlap(dY, rows, Y, rows, K, dtype, true)))
        return MOEGG_EINVAL;
    moegg::SpreadParams p = {};
    p.src = dOut;
    p.other = dw ? Y : nullptr;
    p.map = row_map;
    p.weights = topk_weights;
    p.offsets = offsets;
    p.padded = padded_offsets;
    p.map_is_padded = true;
    p.dst = dY;
    p.dw = dw;
    p.err = error_flags;
    p.T = num_tokens;
    p.rows = rows;
    p.topk = topk;
    p.E = num_experts;
    p.K = K;
    return from_hip(moegg::spread_launch(p, dtype, static_cast<hipStream_t>(stream)));
}

// Sizes of the adapter entry points; also bounds every launch's grid.
static moegg_status check_lora_sizes(int64_t T, int32_t L, int32_t R, int32_t K, int32_t N)
{
    constexpr int64_t kMax = (int64_t)1 << 39;  // elements: 2^40 bytes of 16 bits
    if (T < 0 || T > INT32_MAX || L < 1 || L > MOEGG_MAX_EXPERTS || R < 1 ||
        R > MOEGG_MAX_LORA_RANK || K < 8 || N < 8 || K > (1 << 30) || N > (1 << 30))
        return MOEGG_ESHAPE;
    const int64_t wide = K > N ? K : N;
    if ((int64_t)L * R > kMax / wide || (T > 0 && wide > kMax / T))
        return MOEGG_ESHAPE;
    // Launch sizes: shrink's workgroups have 512 threads, the others 256;
    // expand has at most its places (1024) and one workgroup a tile.
    const int64_t tiles = T / 16 + 1 + L;
    const int wide_splits = moegg::lora_splits(T, L, R, (int32_t)wide);
    const int64_t cols = ((int64_t)K + 127) / 128 + ((int64_t)N + 127) / 128;
    const int64_t grad = (L + T / moegg::lora_chunk(T, R, K, N)) * cols * ((R + 15) / 16);
    if (tiles * wide_splits >= kMaxThreads / 512 || tiles + 1024 >= kMaxThreads / 256 ||
        grad >= kMaxThreads / 256)
        return MOEGG_ESHAPE;
    return MOEGG_OK;
}

// Row stride of a matrix of T rows of n elements.
static bool stride_ok(int64_t ld, int64_t n, int64_t T)
{
    return ld >= n && ld <= INT32_MAX && (T == 0 || ld <= ((int64_t)1 << 39) / T);
}

// Whether two matrices of T rows of 16-bit elements share any.  With one row
// stride (column slices of one matrix, say) columns and rows decide; with two
// any common stretch of memory counts.
static bool rows_overlap(const void *a, int64_t ld_a, int64_t cols_a, const void *b, int64_t ld_b,
                         int64_t cols_b, int64_t T)
{
    if (!a || !b || T == 0)
        return false;
    const int64_t pa = reinterpret_cast<intptr_t>(a), pb = reinterpret_cast<intptr_t>(b);
    const int64_t end_a = pa + 2 * ((T - 1) * ld_a + cols_a);
    const int64_t end_b = pb + 2 * ((T - 1) * ld_b + cols_b);
    if (pa >= end_b || pb >= end_a)
        return false;
    if (ld_a != ld_b)
        return true;
    const int64_t row = 2 * ld_a;
    const int64_t shift = ((pb - pa) % row + row) % row;  // b's first column in a's rows
    return shift < 2 * cols_a || shift + 2 * cols_b > row;
}

static size_t lora_h_bytes(int64_t T, int32_t L, int32_t R, int32_t C)
{
    // 32 bytes behind the last row: it is read in pieces of 8 values
    const size_t b = (size_t)moegg::lora_splits(T, L, R, C) * (size_t)T * (size_t)R * sizeof(float);
    return T > 0 ? (b + 32 + 255) / 256 * 256 : 0;
}

// dh summed over the splits, for the weight gradients.
static size_t lora_sum_bytes(int64_t T, int32_t L, int32_t R, int32_t C)
{
    const size_t b = (size_t)T * (size_t)R * sizeof(float);
    return moegg::lora_splits(T, L, R, C) > 1 ? (b + 255) / 256 * 256 : 0;
}

size_t moegg_lora_workspace_bytes(int64_t num_rows, int32_t num_adapters, int32_t R, int32_t K,
                                  int32_t N)
{
    if (check_lora_sizes(num_rows, num_adapters, R, K, N) != MOEGG_OK)
        return 0;
    return lora_h_bytes(num_rows, num_adapters, R, K);
}

size_t moegg_lora_bwd_workspace_bytes(int64_t num_rows, int32_t num_adapters, int32_t R,
                                      int32_t K, int32_t N)
{
    if (check_lora_sizes(num_rows, num_adapters, R, K, N) != MOEGG_OK)
        return 0;
    // dh (and its sum over splits), then the chunks' partial sums: adapters of more than one chunk hold
    // fewer than 2 T / chunk of them together
    const int64_t chunk = moegg::lora_chunk(num_rows, R, K, N);
    const size_t parts = num_rows > chunk ? (size_t)(2 * num_rows / chunk) : 0;
    return lora_h_bytes(num_rows, num_adapters, R, N) +
           lora_sum_bytes(num_rows, num_adapters, R, N) +
           parts * (size_t)R * ((size_t)K + (size_t)N) * sizeof(float);
}

static moegg_status check_lora_dtype(int32_t dtype)
{
    return !known_dtype(dtype) ? MOEGG_EINVAL : dtype == MOEGG_FP32 ? MOEGG_EUNSUPPORTED : MOEGG_OK;
}

// all_rows: rows of no adapter get base's row; otherwise they keep what Y holds.
static moegg_status lora_fwd(const void *X, int64_t ldx, const void *A, const void *B, const int32_t
                             *m_sizes, const int32_t *gather_idx, const int32_t *ranks, const float
                             *scales, int32_t dtype, int64_t num_rows, int32_t num_adapters, int32_t
                             R, int32_t K, int32_t N, const void *base, int64_t ld_base, void *Y,
                             int64_t ldy, float *H, void *workspace, size_t workspace_bytes, int32_t
                             *error_flags, void *stream, bool all_rows)
{
    moegg_status st = check_lora_sizes(num_rows, num_adapters, R, K, N);
    if (st == MOEGG_OK)
        st = check_lora_dtype(dtype);
    if (st != MOEGG_OK)
        return st;
    if (!base) {
        base = Y;
        ld_base = ldy;
    }
    if (!stride_ok(ldx, K, num_rows) || !stride_ok(ldy, N, num_rows) ||
        !stride_ok(ld_base, N, num_rows))
        return MOEGG_ESHAPE;
    if (num_rows == 0)
        return MOEGG_OK;
    if (!X || !A || !B || !m_sizes || !Y || !aligned2(X) || !aligned2(A) || !aligned2(B) ||
        !aligned4(m_sizes) || !aligned4(gather_idx) || !aligned4(ranks) || !aligned4(scales) ||
        !aligned2(base) || !aligned2(Y) || !aligned4(H) || (base == Y && ld_base != ldy))
        return MOEGG_EINVAL;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < moegg_lora_workspace_bytes(num_rows, num_adapters, R, K, N))
        return MOEGG_EWORKSPACE;
    moegg::LoraParams p = {};
    p.m_sizes = m_sizes;
    p.gather = gather_idx;
    p.ranks = ranks;
    p.scales = scales;
    p.err = error_flags;
    p.T = num_rows;
    p.L = num_adapters;
    p.R = R;
    p.splits = moegg::lora_splits(num_rows, num_adapters, R, K);
    p.split_stride = num_rows * R;
    p.h = static_cast<float *>(workspace);
    p.in = static_cast<const uint16_t *>(X);
    p.w = static_cast<const uint16_t *>(A);
    p.ld_in = ldx;
    p.C = K;
    hipError_t e = moegg::lora_shrink_launch(p, dtype, false, static_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return from_hip(e);
    p.w = static_cast<const uint16_t *>(B);
    p.C = N;
    p.base = static_cast<const uint16_t *>(base);
    p.out = static_cast<uint16_t *>(Y);
    p.ld_base = ld_base;
    p.ld_out = ldy;
    p.stream_base = moegg::lora_streams(num_rows, N);
    p.copy_unrouted = all_rows && base != Y;
    p.h_out = H;
    return from_hip(
        moegg::lora_expand_launch(p, dtype, false, static_cast<hipStream_t>(stream)));
}

moegg_status moegg_lora_fwd(const void *X, int64_t ldx, const void *A, const void *B,
                            const int32_t *m_sizes, const int32_t *gather_idx,
                            const int32_t *ranks, const float *scales, int32_t dtype,
                            int64_t num_rows, int32_t num_adapters, int32_t R, int32_t K,
                            int32_t N, const void *base, int64_t ld_base, void *Y, int64_t ldy,
                            float *H, void *workspace, size_t workspace_bytes,
                            int32_t *error_flags, void *stream)
{
    return lora_fwd(X, ldx, A, B, m_sizes, gather_idx, ranks, scales, dtype, num_rows, num_adapters,
                    R, K, N, base, ld_base, Y, ldy, H, workspace, workspace_bytes, error_flags,
                    stream, false);
}

moegg_status moegg_lora_fwd_all_rows(const void *X, int64_t ldx, const void *A, const void *B, const
                                     int32_t *m_sizes, const int32_t *gather_idx, const int32_t
                                     *ranks, const float *scales, int32_t dtype, int64_t num_rows,
                                     int32_t num_adapters, int32_t R, int32_t K, int32_t N, const
                                     void *base, int64_t ld_base, void *Y, int64_t ldy, float *H,
                                     void *workspace, size_t workspace_bytes, int32_t *error_flags,
                                     void *stream)
{
    return lora_fwd(X, ldx, A, B, m_sizes, gather_idx, ranks, scales, dtype, num_rows, num_adapters,
                    R, K, N, base, ld_base, Y, ldy, H, workspace, workspace_bytes, error_flags,
                    stream, true);
}

moegg_status moegg_lora_bwd(const void *X, int64_t ldx, const void *dY, int64_t lddy,
                            const void *A, const void *B, const float *H, const int32_t *m_sizes,
                            const int32_t *gather_idx, const int32_t *ranks, const float *scales,
                            int32_t dtype, int64_t num_rows, int32_t num_adapters, int32_t R,
                            int32_t K, int32_t N, const void *base, int64_t ld_base, void *dX,
                            int64_t lddx, void *dA, void *dB, uint32_t flags, void *workspace,
                            size_t workspace_bytes, int32_t *error_flags, void *stream)
{
    moegg_status st = check_lora_sizes(num_rows, num_adapters, R, K, N);
    if (st == MOEGG_OK)
        st = check_lora_dtype(dtype);
    if (st != MOEGG_OK)
        return st;
    if (!dA != !dB || (flags & ~(uint32_t)(MOEGG_LORA_FP32_GRAD | MOEGG_LORA_ALL_ROWS)))
        return MOEGG_EINVAL;
    if (!dX)
        lddx = K;
    if (!base || !dX) {
        base = dX;
        ld_base = lddx;
    }
    if (!dA)
        ldx = K;
    if (!stride_ok(ldx, K, num_rows) || !stride_ok(lddy, N, num_rows) ||
        !stride_ok(lddx, K, num_rows) || !stride_ok(ld_base, K, num_rows))
        return MOEGG_ESHAPE;
    if (num_rows == 0 && !dA)
        return MOEGG_OK;
    if (!m_sizes || !aligned4(m_sizes) || !aligned4(gather_idx) || !aligned4(ranks) ||
        !aligned4(scales) || !aligned2(base) || !aligned2(dX) || (base == dX && ld_base != lddx))
        return MOEGG_EINVAL;
    if (num_rows > 0 && (!dY || !A || !B || !aligned2(dY) || !aligned2(A) || !aligned2(B)))
        return MOEGG_EINVAL;
    if (dA) {
        if (num_rows > 0 && (!X || !H || !aligned2(X) || !aligned4(H)))
            return MOEGG_EINVAL;
        // dX is written before X is read for dA and dY for dB
        if (rows_overlap(dX, lddx, K, X, ldx, K, num_rows) ||
            rows_overlap(dX, lddx, K, dY, lddy, N, num_rows))
            return MOEGG_EINVAL;
        if ((flags & MOEGG_LORA_FP32_GRAD) ? !aligned4(dA) || !aligned4(dB)
                                           : !aligned2(dA) || !aligned2(dB))
            return MOEGG_EINVAL;
    }
    if (num_rows > 0 &&
        (!workspace || !aligned16(workspace) ||
         workspace_bytes < moegg_lora_bwd_workspace_bytes(num_rows, num_adapters, R, K, N)))
        return MOEGG_EWORKSPACE;
    moegg::LoraParams p = {};
    p.m_sizes = m_sizes;
    p.gather = gather_idx;
    p.ranks = ranks;
    p.scales = scales;
    p.err = error_flags;
    p.T = num_rows;
    p.L = num_adapters;
    p.R = R;
    p.splits = moegg::lora_splits(num_rows, num_adapters, R, N);
    p.split_stride = num_rows * R;
    p.h = static_cast<float *>(workspace);
    p.scale_shrink = true;
    p.in = static_cast<const uint16_t *>(dY);
    p.w = static_cast<const uint16_t *>(B);
    p.ld_in = lddy;
    p.C = N;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t e = moegg::lora_shrink_launch(p, dtype, true, hs);
    // dh for the weight gradients: dX's launch adds the splits on its way.
    char *const after_h = static_cast<char *>(workspace) + lora_h_bytes(num_rows, num_adapters, R, N);
    const bool split = num_rows > 0 && p.splits > 1;
    float *const dh = split ? reinterpret_cast<float *>(after_h) : p.h;
    if (e == hipSuccess && dX) {
        p.w = static_cast<const uint16_t *>(A);
        p.C = K;
        p.base = static_cast<const uint16_t *>(base);
        p.out = static_cast<uint16_t *>(dX);
        p.ld_base = ld_base;
        p.ld_out = lddx;
        p.stream_base = moegg::lora_streams(num_rows, K);
        p.copy_unrouted = (flags & MOEGG_LORA_ALL_ROWS) && base != dX;
        p.h_out = dA && split ? dh : nullptr;
        e = moegg::lora_expand_launch(p, dtype, true, hs);
    } else if (e == hipSuccess && split) {
        e = moegg::lora_sum_launch(p.h, dh, num_rows * R, p.splits, hs);
    }
    if (e != hipSuccess || !dA)
        return from_hip(e);
    moegg::GradParams g = {};
    g.l = p;
    g.x = static_cast<const uint16_t *>(X);
    g.dy = static_cast<const uint16_t *>(dY);
    g.h = H;
    g.dh = dh;
    g.dA = dA;
    g.dB = dB;
    g.partials = reinterpret_cast<float *>(after_h + lora_sum_bytes(num_rows, num_adapters, R, N));
    g.ld_x = ldx;
    g.ld_dy = lddy;
    g.R = R;
    g.K = K;
    g.N = N;
    g.chunk = moegg::lora_chunk(num_rows, R, K, N);
    g.col_tiles_a = (K + 127) / 128;
    g.col_tiles_b = (N + 127) / 128;
    g.fp32_out = flags & MOEGG_LORA_FP32_GRAD;
    return from_hip(moegg::lora_grad_launch(g, dtype, hs));
}

}  // extern "C"
