/*
 * moegg.h -- MoE grouped GEMM for AMD Instinct MI355X (gfx950).
 *
 * C ABI of libmoegg.so: expert routing metadata, the forward grouped GEMM
 * with its gather / scatter / gate-multiply fusions, its two backward
 * GEMMs, and a launch of explicit GEMM groups of different shapes.
 *
 * Conventions shared by every entry point
 *   T = num_tokens, k = topk, S = T * k routed slots; slot s = t * k + j is
 *   the j-th expert choice of token t (row-major [T, k] order).
 *   E = num_experts.  W is [E, N, K] row-major (K contiguous), the layout of
 *   grouped_gemm_forward in unsloth grouped_gemm/interface.py.
 *   bf16 tensors are row-major, 2 bytes per element; base pointers must be
 *   2-byte aligned (fp32 outputs 4-byte).  Any K and N are accepted: when
 *   every row of a call is whole 16-byte chunks (K and N multiples of 8 and
 *   operands 16-byte aligned) the tiled kernels run, otherwise slower
 *   any-shape kernels that compute the same definitions (no workspace;
 *   workspace arguments are then ignored and the workspace size queries
 *   return 0 for such K and N).
 *   Each input operand (X, dY, one expert's W, a group's x or w) must be
 *   smaller than 2 GiB: the kernels address them with 32-bit offsets.
 *   Index tensors are int32.  "sorted position" p indexes the expert-grouped
 *   order: expert e owns positions [off[e], off[e] + m_sizes[e]).
 *
 * Ownership and ordering
 *   Every pointer is a device pointer owned by the caller (unless stated as
 *   a host pointer).  The library never allocates, frees or synchronises;
 *   each call enqueues its kernels on `stream` (a hipStream_t; NULL is the
 *   default stream) and returns.  Calls on one stream run in order.
 *   Every element of every output is written by the call (the caller need
 *   not clear outputs), except rows that belong to dropped slots.
 *
 * Errors
 *   Host-checkable preconditions (the asserts of the pages' launchers)
 *   return a status before anything is enqueued.  Data-dependent problems
 *   found on the device (an expert id outside [0, E), m_sizes that are
 *   negative or sum past S, a gather index outside [0, S)) are ORed as
 *   MOEGG_DERR_* bits into *error_flags when that pointer is non-NULL; the
 *   kernels skip the offending rows instead of faulting.  *error_flags is
 *   sticky: the library never clears it.
 */
#ifndef MOEGG_H
#define MOEGG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOEGG_OK = 0,
    MOEGG_EINVAL = 1,       /* illegal flag combination or missing pointer       */
    MOEGG_ESHAPE = 2,       /* non-positive, misaligned or inconsistent sizes     */
    MOEGG_EUNSUPPORTED = 3, /* legal on the pages but not offered here            */
    MOEGG_EWORKSPACE = 4,   /* workspace missing or smaller than required         */
    MOEGG_EHIP = 5          /* a HIP launch or query failed                       */
} moegg_status;

/* Flags: the pages' fusion switches (grouped_gemm_forward arguments). */
#define MOEGG_PERMUTE_X 1u     /* gather X rows from token order on load          */
#define MOEGG_PERMUTE_Y 2u     /* scatter output rows back to slot order on store */
#define MOEGG_FUSE_MUL_POST 4u /* multiply each output row by its gate weight     */
#define MOEGG_DW_FP32_OUT 8u   /* dW only: write fp32 instead of bf16             */
#define MOEGG_GATED_SILU 32u   /* forward only: gated SiLU on (gate, linear) pairs */
#define MOEGG_GATED_GELU 64u   /* i8 and gated entry points: gated GELU (tanh form)  */
#define MOEGG_GATED_HALVES 128u /* the same: gate rows, then linear rows, no pairs  */

/* Device error bits ORed into *error_flags. */
#define MOEGG_DERR_EXPERT_ID 1 /* a top-k expert id outside [0, E): slot dropped  */
#define MOEGG_DERR_M_SIZES 2   /* m_sizes negative or summing past S: clipped     */
#define MOEGG_DERR_GATHER 4    /* a gather index outside [0, S): row skipped      */
#define MOEGG_DERR_LOGIT 8     /* a gate logit or bias NaN or +inf: expert masked */
#define MOEGG_DERR_RANK 16     /* an adapter's rank outside [0, R]: clipped       */

#define MOEGG_MAX_EXPERTS 1024
#define MOEGG_MAX_GROUPS 16
#define MOEGG_MAX_TOPK 64       /* moegg_gate: picks a token                       */
#define MOEGG_MAX_GATE_GROUPS 64
#define MOEGG_MAX_LORA_RANK 256
#define MOEGG_MAX_I8_K 131056   /* moegg_grouped_gemm_i8: 128 * 128 * K stays in int32 */

/* Element types of the entry points that take a dtype. */
#define MOEGG_BF16 0
#define MOEGG_FP16 1
#define MOEGG_FP32 2

/* Human-readable name of a status code (static string). */
const char *moegg_status_string(moegg_status status);

/* Library ABI version (major * 100 + minor). */
int32_t moegg_version(void);

/*
 * Bytes of device workspace moegg_route needs for num_slots = T * k slots
 * and num_experts experts (per-chunk expert counts).  0 for num_slots = 0.
 */
size_t moegg_route_workspace_bytes(int64_t num_slots, int32_t num_experts);

/*
 * moegg_route -- expert histogram, offsets and stable gather/scatter indices.
 *
 * Follows the routing metadata the pages consume: m_sizes (the per-expert
 * slot counts of the grouped_gemm_forward docstring,
 * grouped_gemm/interface.py), expt_hist and its cumsum offsets, the
 * block-padded layout of the ragged dw comment block, and GatherIndx /
 * ScatterIndx in triton_kernels/matmul_ogs.py, where the scatter index is
 * the inverse permutation of the gather index.
 *
 *   topk_ids       [S] int32, slot order (the router's [T, k] ids).
 *   m_sizes        out [E]   number of slots routed to each expert.
 *   offsets        out [E+1] exclusive prefix sum of m_sizes.
 *   padded_offsets out [E+1] the same with each count rounded up to a
 *                  multiple of block_m; may be NULL.
 *   tile_offsets   out [E+1] exclusive prefix sum of ceil(m_sizes/block_m);
 *                  may be NULL.
 *   gather_idx     out [S] slot held at sorted position p.  Within an expert,
 *                  slots appear in ascending order (a stable sort).
 *   scatter_idx    out [S] sorted position of slot s (the inverse of
 *                  gather_idx); may be NULL.
 *   workspace      device scratch of moegg_route_workspace_bytes(S, E) bytes,
 *                  contents need no initialisation.
 *
 * A slot whose id is outside [0, E) is dropped: scatter_idx = -1, the
 * positions it would have used stay at the end with gather_idx = -1, and
 * MOEGG_DERR_EXPERT_ID is raised.  Results are bit-for-bit deterministic.
 * Errors: ESHAPE if T < 0, k < 1, E < 1, E > MOEGG_MAX_EXPERTS or
 * block_m < 1; EINVAL for a NULL required pointer; EWORKSPACE if
 * workspace_bytes is too small.  T = 0 writes zero histograms and offsets.
 */
moegg_status moegg_route(const int32_t *topk_ids, int32_t num_tokens, int32_t topk,
                         int32_t num_experts, int32_t block_m, int32_t *m_sizes,
                         int32_t *offsets, int32_t *padded_offsets, int32_t *tile_offsets,
                         int32_t *gather_idx, int32_t *scatter_idx, void *workspace,
                         size_t workspace_bytes, int32_t *error_flags, void *stream);

/* Size of the device array moegg_route_noalloc keeps its counts in. */
#define MOEGG_ROUTE_NOALLOC_MAX_BYTES (1u << 20)

/*
 * moegg_route_noalloc -- moegg_route without a workspace, for callers that
 * cannot allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  It calls no allocating routine.
 *
 * The per-chunk counts go to a static device array of
 * MOEGG_ROUTE_NOALLOC_MAX_BYTES bytes that the library holds on every device
 * it runs on until the process ends (its address is looked up on the first
 * call on each device).  A call with moegg_route_workspace_bytes(T * topk, E)
 * larger than that (e.g. more than 65,536 slots with E = 1024, or more than
 * 2^21 slots with E = 32) returns MOEGG_EWORKSPACE before anything is
 * enqueued.  All calls on one device share the array: calls that may run at
 * the same time on that GPU (streams without ordering between them) race and
 * give wrong results; calls ordered on one stream do not, since each call
 * writes every count it reads.  Otherwise the same arguments, results and
 * errors as moegg_route.
 */
moegg_status moegg_route_noalloc(const int32_t *topk_ids, int32_t num_tokens, int32_t topk,
                                 int32_t num_experts, int32_t block_m, int32_t *m_sizes,
                                 int32_t *offsets, int32_t *padded_offsets, int32_t *tile_offsets,
                                 int32_t *gather_idx, int32_t *scatter_idx, int32_t *error_flags,
                                 void *stream);

/*
 * moegg_grouped_gemm_fwd -- Y_e = X_e W_e^T for every expert, one launch.
 *
 * grouped_gemm_forward (grouped_gemm/interface.py) and the per-expert loop
 * of matmul_ogs_torch (triton_kernels/matmul_ogs.py).  For sorted position p
 * of expert e, with fp32 accumulation:
 *   y[n] = sum_k X[src(p), k] * W[e, n, k]
 *   src(p) = gather_idx[p] / topk with MOEGG_PERMUTE_X (X is [T, K], token
 *            order), else p (X is [S, K], already in expert order);
 *   MOEGG_FUSE_MUL_POST: y *= topk_weights[gather_idx[p]] (fp32 gate of the
 *            slot, topk_weights is [S] in slot order);
 *   stored as bf16 (round to nearest even) to row gather_idx[p] of Y with
 *   MOEGG_PERMUTE_Y, else to row p.  Y is [S, N].
 *   MOEGG_GATED_SILU: the gate_up GEMM with its activation fused (the
 *            FusedActivation of triton_kernels/matmul_ogs.py with
 *            reduction_n = 2, output width N/2).  W rows come in adjacent
 *            (gate, linear) pairs and
 *              out[c] = silu(y[2c]) * y[2c + 1],  silu(x) = x / (1 + e^-x),
 *            from the fp32 accumulators, rounded once to bf16.  Y is
 *            [S, N/2].  Not with PERMUTE_Y or FUSE_MUL_POST (the activation
 *            belongs to the first GEMM); N must be even.
 *
 *   m_sizes     [E] device int32 rows per expert (moegg_route output); read
 *               on the device, no host synchronisation.
 *   gather_idx  [S] device int32; required with either permute flag.
 *   error_flags optional device int32 (see Errors above).
 *
 * Errors: EINVAL if both permute flags are set, FUSE_MUL_POST without
 * PERMUTE_Y, GATED_SILU with PERMUTE_Y or FUSE_MUL_POST, an unknown flag, or
 * a required pointer is NULL (gather_idx with a permute flag, topk_weights
 * with FUSE_MUL_POST); ESHAPE for non-positive sizes, odd N with
 * GATED_SILU, E > MOEGG_MAX_EXPERTS, a pointer that is not 2-byte aligned.
 * T = 0 is a no-op.
 */
moegg_status moegg_grouped_gemm_fwd(const void *X, const void *W, const int32_t *m_sizes,
                                    const int32_t *gather_idx, const float *topk_weights,
                                    int32_t num_tokens, int32_t topk, int32_t num_experts,
                                    int32_t N, int32_t K, uint32_t flags, void *Y,
                                    int32_t *error_flags, void *stream);

/*
 * moegg_grouped_gemm_dX -- dX_e = dY_e W_e (reduction over N), one launch.
 *
 * grouped_gemm_dX (grouped_gemm/interface.py).  `flags` are the permute
 * flags the forward used:
 *   dY row     q(p) = gather_idx[p] if the forward used PERMUTE_Y (dY is in
 *              slot order and is gathered on load), else p;
 *   dX[., k]   = sum_n dY[q(p), n] * W[e, n, k]   (fp32 accumulation)
 *   stored bf16 to row gather_idx[p] if the forward used PERMUTE_X (scatter
 *   back to slot order), else row p.  dY is [S, N], dX is [S, K]; summing a
 *   token's top-k rows is left to the caller.
 *
 * Tail balancing (optional): a persistent launch runs its tiles in rounds
 * of one tile per workgroup.  With a workspace, the tiles of a last, partial
 * round have their reductions over N cut into parts spread over the
 * otherwise idle workgroups (the split-k of triton_kernels/matmul_ogs.py,
 * fp32 partials summed by a separate launch), summed in part order:
 * deterministic, and equal to the unsplit result up to fp32 rounding order.
 *   workspace       device, 16-byte aligned, at least
 *                   moegg_grouped_gemm_dX_workspace_bytes(...) bytes (no
 *                   initialisation needed), or NULL: no split.
 *   workspace_bytes its size; 0 with NULL.
 * Errors: EINVAL for both permute flags or a missing gather_idx;
 * EUNSUPPORTED for FUSE_MUL_POST (the pages forbid it in training);
 * ESHAPE as for the forward; EWORKSPACE for a workspace smaller than needed.
 */
moegg_status moegg_grouped_gemm_dX(const void *dY, const void *W, const int32_t *m_sizes,
                                   const int32_t *gather_idx, int32_t num_tokens, int32_t topk,
                                   int32_t num_experts, int32_t N, int32_t K, uint32_t flags,
                                   void *dX, void *workspace, size_t workspace_bytes,
                                   int32_t *error_flags, void *stream);

/*
 * Bytes of workspace moegg_grouped_gemm_dX can use to balance its last
 * round of tiles, for these sizes on the current device (it depends on the
 * device's compute units): a small header plus fp32 partials of at most one
 * tile per workgroup of the launch.  0 if the sizes are invalid or the
 * device cannot be queried.
 */
size_t moegg_grouped_gemm_dX_workspace_bytes(int32_t num_tokens, int32_t topk,
                                             int32_t num_experts, int32_t N, int32_t K);

/*
 * moegg_grouped_gemm_dW -- dW_e = dY_e^T X_e, a reduction over each expert's
 * own (ragged) number of rows, one launch.
 *
 * grouped_gemm_dW (grouped_gemm/interface.py) and the ragged-K formulation of
 * triton_kernels/matmul_ogs.py, which computes dw as a grouped matmul of x
 * transposed with dy:
 *   dW[e, n, k] = sum_{p in e} dY[q(p), n] * X[r(p), k]  (fp32 accumulation)
 *   r(p) = gather_idx[p] / topk with PERMUTE_X (X is [T, K]), else p
 *   (X is [S, K]); q(p) = gather_idx[p] with PERMUTE_Y, else p.
 * dW is [E, N, K], bf16, or fp32 with MOEGG_DW_FP32_OUT.  Experts with no
 * rows get exact zeros.
 *
 * Short launches (S <= 1024 and S <= 16 * num_experts, each operand below
 * 1 GiB, e.g. a decode step) run a kernel whose cost is its output stores:
 * no split and no gather copy, so any workspace is left unused.
 *
 * Split reduction (the split-k of triton_kernels/matmul_ogs.py, whose fp32
 * partials a separate reduce sums, applied to the rows of hot experts):
 * with a workspace, an expert holding many more rows than the average is
 * cut into chunks of rows whose fp32 partial products go to the workspace;
 * a second launch on the same stream sums each expert's partials in chunk
 * order and writes its dW.  The result is deterministic (the same for every
 * run with the same inputs and workspace size), and differs from the
 * unsplit sum only by fp32 rounding order.
 *   workspace       device, 16-byte aligned, of at least
 *                   moegg_grouped_gemm_dW_workspace_bytes(...) bytes
 *                   (contents need no initialisation), or NULL: no split.
 *   workspace_bytes its size; 0 with NULL.
 * Errors: as for dX; EWORKSPACE if a workspace is given but smaller than
 * needed.
 */
moegg_status moegg_grouped_gemm_dW(const void *X, const void *dY, const int32_t *m_sizes,
                                   const int32_t *gather_idx, int32_t num_tokens, int32_t topk,
                                   int32_t num_experts, int32_t N, int32_t K, uint32_t flags,
                                   void *dW, void *workspace, size_t workspace_bytes,
                                   int32_t *error_flags, void *stream);

/*
 * Bytes of workspace moegg_grouped_gemm_dW can use to split hot experts'
 * reductions, for these sizes: a small header plus fp32 [N, K] partials for
 * fewer than 2 S / split_rows chunks, where split_rows is about
 * S * ceil(N/256) * ceil(K/256) / 768 rows (at least 256).  0 when no
 * expert can hold more than split_rows rows, or when S <= 1024 (reductions
 * that short are never split); the workspace is then unused.
 */
size_t moegg_grouped_gemm_dW_workspace_bytes(int32_t num_tokens, int32_t topk,
                                             int32_t num_experts, int32_t N, int32_t K);

/*
 * Bytes of workspace with which moegg_grouped_gemm_dW under MOEGG_PERMUTE_X
 * also copies X's rows into expert order before the reduction: the split
 * area above rounded up to 256 bytes, plus S * K * 2 for the copy.  The copy
 * (X[gather_idx[p] / topk, :] for every sorted position p below the sum of
 * m_sizes) is a separate launch on the same stream; the reduction then
 * reads it in sorted order.  The result is the same as with the gather
 * inside the reduction, including zeros and MOEGG_DERR_GATHER for entries
 * outside [0, S); positions past the sum of m_sizes, where routing leaves
 * its dropped slots, are read by neither.  On MI355X the copy plus the
 * reduction take less time.  The copy is an operand like X and must stay
 * below 2 GiB: when S * K * 2 >= 2^31, or for a short launch (see
 * moegg_grouped_gemm_dW), this returns moegg_grouped_gemm_dW_workspace_bytes(...)
 * and moegg_grouped_gemm_dW gathers inside the reduction whatever the
 * workspace size.  A workspace of
 * at least moegg_grouped_gemm_dW_workspace_bytes(...) bytes but less than
 * this keeps the gather inside the reduction.  Without MOEGG_PERMUTE_X the
 * extra bytes are unused.
 */
size_t moegg_grouped_gemm_dW_gather_workspace_bytes(int32_t num_tokens, int32_t topk,
                                                    int32_t num_experts, int32_t N, int32_t K);

/*
 * One GEMM group: y[m, n] = x[m, k] @ w, bf16 in, fp32 accumulation, bf16 out.
 * w is [k, n] row-major (ldw >= n) when the call's trans_b is 0, as in
 * asym_dual_gmm_separated (wall_x/fusions/backend.py), or [n, k] row-major
 * (ldw >= k) when trans_b is 1.  Leading dimensions are in elements.
 */
typedef struct {
    const void *x;
    const void *w;
    void *y;
    int32_t m, n, k;
    int32_t ldx, ldw, ldy;
} moegg_group;

/*
 * moegg_grouped_gemm_groups -- several independent GEMMs of different shapes
 * in one launch: the asymmetric dual-expert GEMM of asym_dual_gmm_separated
 * (wall_x/fusions/backend.py), which multiplies each expert's own input by
 * its own weight and computes both products in one fused call.
 *
 *   groups      HOST array of num_groups descriptors (copied at launch; it
 *               may be freed when the call returns).  1 <= num_groups <=
 *               MOEGG_MAX_GROUPS.  A group with m = 0 is skipped.
 *   trans_b     0: w is [k, n]; 1: w is [n, k].  trans_a is not offered
 *               (inputs are [m, k]).
 * Errors: EINVAL for a NULL pointer or bad trans_b; ESHAPE for negative
 * sizes, a pointer that is not 2-byte aligned, or a leading dimension
 * smaller than its row.
 */
moegg_status moegg_grouped_gemm_groups(const moegg_group *groups, int32_t num_groups,
                                       int32_t trans_b, void *stream);

/* Combine flag: write the combine's output in fp32 instead of bf16. */
#define MOEGG_COMBINE_FP32_OUT 16u

/*
 * moegg_combine -- the top-k combine after the second grouped GEMM: each
 * token's k expert outputs, weighted by their routing probabilities and
 * summed.  This is the unpermute of wall_x/fusions/backend.py (expert outputs
 * back to token order, combined with the routing probabilities) and the
 * n_expts_act reduction at the end of matmul_ogs in
 * triton_kernels/matmul_ogs.py (matmul_ogs_torch accumulates it in fp32):
 *
 *   out[t, n] = sum_{j<k} w[t*k + j] * Y[row(t*k + j), n]   (fp32, j ascending)
 *
 *   Y              [y_rows, N] bf16 device, row-major.
 *   scatter_idx    [T*k] int32 device: row of Y holding slot s (moegg_route's
 *                  scatter_idx when Y is in expert-sorted order); a negative
 *                  entry is a dropped slot and adds nothing.  NULL: Y is in
 *                  slot order (the PERMUTE_Y output), row(s) = s, and
 *                  y_rows >= T*k.
 *   topk_weights   [T*k] fp32 device, slot order, or NULL for weight 1 (the
 *                  rows already carry the gates, as after FUSE_MUL_POST).
 *   flags          0 or MOEGG_COMBINE_FP32_OUT.
 *   out            [T, N] device, bf16 (rounded once from the fp32 sum) or
 *                  fp32.  Every element is written.
 *   error_flags    optional device int32; an entry of scatter_idx at or above
 *                  y_rows sets MOEGG_DERR_GATHER and the slot is skipped.
 * Any N; Y and out 2-byte aligned (out 4-byte for fp32).  T = 0 is a no-op.
 * Errors: ESHAPE for bad sizes, EINVAL for unknown flags, NULL or misaligned
 * pointers.
 */
moegg_status moegg_combine(const void *Y, const int32_t *scatter_idx, const float *topk_weights,
                           int64_t num_tokens, int32_t topk, int32_t N, int64_t y_rows,
                           uint32_t flags, void *out, int32_t *error_flags, void *stream);

/*
 * moegg_combine_bwd -- backward of moegg_combine (unpermute_bwd,
 * wall_x/fusions/backend.py, which takes the forward input so that the
 * routing probabilities get a gradient as well):
 *
 *   dY[row(s), n] = w[s] * dOut[t, n]                    (rounded to bf16)
 *   dw[s]         = sum_n dOut[t, n] * Y[row(s), n]      (fp32)
 *
 * for s = t*k + j, with row() and w as in moegg_combine (w = 1 when
 * topk_weights is NULL).
 *   dOut   [T, N] bf16 device.
 *   Y      the forward's input [y_rows, N] bf16; read only when dw != NULL.
 *   dY     [y_rows, N] bf16 device; only rows some slot maps to are written
 *          (all of them when scatter_idx is a permutation or NULL).
 *   dw     [T*k] fp32 device, or NULL to skip the weight gradient.  A dropped
 *          slot gets dw = 0 and writes no dY row.
 * Alignment, sizes and errors as moegg_combine.
 */
moegg_status moegg_combine_bwd(const void *dOut, const void *Y, const int32_t *scatter_idx,
                               const float *topk_weights, int64_t num_tokens, int32_t topk,
                               int32_t N, int64_t y_rows, void *dY, float *dw,
                               int32_t *error_flags, void *stream);

/* Gate flags. */
#define MOEGG_GATE_SIGMOID 1u /* scores are sigmoids of the logits, not their softmax   */
#define MOEGG_GATE_RENORM 2u  /* weights are divided by the sum of the picked scores    */

/*
 * moegg_gate -- from router logits to each token's top-k expert ids and
 * weights: the step in front of moegg_route, whose topk_ids these ids are
 * (and the topk_weights of the GEMMs and combines, slot order).
 *
 *   score_i = softmax(logits[t])_i, or 1 / (1 + e^-l_i) with GATE_SIGMOID
 *   key_i   = score_i + bias_i (bias 0 when NULL); the topk largest keys are
 *             picked, in falling order, equal keys by rising expert index
 *   w_j     = scale * score_{id_j}; with GATE_RENORM divided by the sum of
 *             the picked scores
 *   n_groups > 1: experts form n_groups groups of E / n_groups neighbours; a
 *             group's value is the sum of its two largest keys (its only key
 *             when one expert is left), and experts are picked inside the
 *             topk_groups groups of largest value (equal values by rising
 *             group index).
 *
 * A logit of -inf masks its expert: score 0, never picked.  So does a bias
 * that is not finite, for the pick alone.  A logit that is NaN or +inf is
 * taken as -inf and raises MOEGG_DERR_LOGIT, as does a bias that is NaN or
 * +inf.  A token with fewer than topk experts left (none, for a padding row
 * of -inf) gets id -1 and weight 0 in the places left over; moegg_route
 * drops those slots (and raises MOEGG_DERR_EXPERT_ID for them).  Scores,
 * weights and sums are fp32; keys with a bias or groups are compared in 64
 * bits, the others by the logits themselves, which give the same order.
 *
 *   logits       [T, E] of `dtype`, rows ld_logits >= E elements apart.
 *   bias         [E] fp32 device, or NULL.
 *   topk_ids     out [T, topk] int32.    topk_weights  out [T, topk] fp32.
 *   scores       out [T, E] fp32, or NULL (a load-balancing loss reads them).
 *                Without bias and groups they may take the logits' place
 *                (fp32, ld_logits = E); any other overlap is EINVAL.
 * T = 0 is a no-op.  Errors: ESHAPE for sizes outside 1 <= E <=
 * MOEGG_MAX_EXPERTS, 1 <= topk <= min(E, MOEGG_MAX_TOPK), 1 <= topk_groups <=
 * n_groups <= MOEGG_MAX_GATE_GROUPS, n_groups dividing E, topk <=
 * topk_groups * E / n_groups, ld_logits >= E; EINVAL for an unknown dtype or
 * flag, a scale that is not finite, NULL or misaligned pointers.
 */
moegg_status moegg_gate(const void *logits, int32_t dtype, int64_t ld_logits, const float *bias,
                        int64_t num_tokens, int32_t num_experts, int32_t topk, int32_t n_groups,
                        int32_t topk_groups, float scale, uint32_t flags, int32_t *topk_ids,
                        float *topk_weights, float *scores, int32_t *error_flags, void *stream);

/*
 * moegg_gate_bwd -- gradient of moegg_gate's weights and scores with respect
 * to the logits, for the ids it picked (the pick itself has no gradient):
 *
 *   dlogits = (d weights / d logits)^T dweights + (d scores / d logits)^T dscores
 *
 *   topk_ids     [T, topk] int32 as moegg_gate wrote them; a negative id has
 *                no gradient, an id >= E none either (MOEGG_DERR_EXPERT_ID).
 *   dweights     [T, topk] fp32.   dscores  [T, E] fp32, or NULL for zero.
 *   dlogits      out [T, E] of `dtype`, contiguous; masked experts get 0.  May
 *                take the logits' place (ld_logits = E; any other overlap is
 *                EINVAL) or that of dscores in fp32.
 * scale and flags as in the forward; the scores are computed again from the
 * logits.  Sums in fp32, one rounding to `dtype`.  Errors as moegg_gate.
 */
moegg_status moegg_gate_bwd(const void *logits, int32_t dtype, int64_t ld_logits,
                            const int32_t *topk_ids, const float *dweights, const float *dscores,
                            int64_t num_tokens, int32_t num_experts, int32_t topk, float scale,
                            uint32_t flags, void *dlogits, int32_t *error_flags, void *stream);

/*
 * moegg_permute -- token rows into expert order, each of a token's topk
 * copies times its weight: Xs[row(s)] = w[s] * X[t] for slot s = t * topk + j.
 *
 *   X              [T, K] of `dtype`, row-major.
 *   scatter_idx    [T*topk] int32, moegg_route's scatter_idx (its entries are
 *                  distinct); negative entries are dropped slots.
 *   topk_weights   [T*topk] fp32 slot order, or NULL for weight 1.
 *   offsets, padded_offsets   moegg_route's, [E+1] int32 each.  Both NULL:
 *                  row(s) = scatter_idx[s].  Both given: the block-padded
 *                  layout, row(s) = scatter_idx[s] - offsets[e] +
 *                  padded_offsets[e] for the slot's expert e, and the pad
 *                  rows between an expert's last row and the next expert's
 *                  first are set to zero.
 *   rows           rows of Xs.  T * topk always suffices without padding,
 *                  T * topk + E * (block_m - 1) with it.
 *   Xs             out [rows, K] of `dtype`.  Rows that no slot maps to and
 *                  that are no pad rows are left as they were.
 *   row_map        out [T*topk] int32: row(s), -1 for a dropped slot.  What
 *                  the other three entry points (and moegg_combine, as its
 *                  scatter_idx) take.  Required in the padded layout, where it
 *                  may not be scatter_idx; optional without (it then repeats
 *                  scatter_idx).
 * A row at or past `rows` raises MOEGG_DERR_GATHER and is skipped.  Products
 * in fp32, rounded once.  T = 0 writes the pad rows alone.
 * Errors: ESHAPE for T < 0 or past 16 million, topk < 1, K < 1, rows < 0,
 * sizes past 2^40 bytes, E outside [1, MOEGG_MAX_EXPERTS] in the padded layout; EINVAL for an unknown
 * dtype, one of offsets / padded_offsets without the other, NULL or
 * misaligned pointers (rows need the alignment of one element only), Xs over
 * X (in these four calls an output overlaps an input's rows only where that is
 * said, and then row for row).
 */
moegg_status moegg_permute(const void *X, int32_t dtype, const int32_t *scatter_idx,
                           const float *topk_weights, const int32_t *offsets,
                           const int32_t *padded_offsets, int64_t num_tokens, int32_t topk,
                           int32_t num_experts, int32_t K, int64_t rows, void *Xs,
                           int32_t *row_map, int32_t *error_flags, void *stream);

/*
 * moegg_permute_bwd -- gradient of moegg_permute:
 *   dX[t] = sum_{j<topk} w[s] * dXs[row_map[s]]   (fp32, j ascending, rounded once)
 *   dw[s] = sum_n X[t, n] * dXs[row_map[s], n]    (fp32), when dw is not NULL
 * X is read only for dw (and may be NULL without it); dX may be X.  A dropped
 * slot adds nothing and gets dw = 0.  Arguments and errors as moegg_permute.
 */
moegg_status moegg_permute_bwd(const void *dXs, int32_t dtype, const void *X,
                               const int32_t *row_map, const float *topk_weights,
                               int64_t num_tokens, int32_t topk, int32_t K, int64_t rows, void *dX,
                               float *dw, int32_t *error_flags, void *stream);

/*
 * moegg_unpermute -- expert-ordered rows back to token order, weighted and
 * summed onto a base (a residual, a shared expert's output):
 *   out[t] = base[t] + sum_{j<topk} w[s] * Y[row_map[s]]
 * in fp32, base first, j ascending, rounded once.  The counterpart of
 * moegg_permute in its three types and its padded layout; moegg_combine is
 * the bf16 form that can write fp32.
 *   Y     [rows, K] of `dtype`.   base  [T, K] of `dtype` or NULL; may be out.
 * Arguments and errors otherwise as moegg_permute.
 */
moegg_status moegg_unpermute(const void *Y, int32_t dtype, const int32_t *row_map,
                             const float *topk_weights, const void *base, int64_t num_tokens,
                             int32_t topk, int32_t K, int64_t rows, void *out,
                             int32_t *error_flags, void *stream);

/*
 * moegg_unpermute_bwd -- gradient of moegg_unpermute (base's is dOut itself):
 *   dY[row_map[s]] = w[s] * dOut[t]                (rounded once; the rows of
 *                                                   row_map are distinct)
 *   dw[s] = sum_n dOut[t, n] * Y[row_map[s], n]    (fp32), when dw is not NULL
 * With offsets and padded_offsets the pad rows of dY are set to zero, so that
 * products over the padded rows read no stale values; other rows no slot maps
 * to are left as they were.  Y is read only for dw; dY may be Y.
 */
moegg_status moegg_unpermute_bwd(const void *dOut, int32_t dtype, const void *Y,
                                 const int32_t *row_map, const float *topk_weights,
                                 const int32_t *offsets, const int32_t *padded_offsets,
                                 int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t K,
                                 int64_t rows, void *dY, float *dw, int32_t *error_flags,
                                 void *stream);

/* Adapter flags. */
#define MOEGG_LORA_FP32_GRAD 1u /* write dA and dB in fp32 instead of `dtype`          */
#define MOEGG_LORA_ALL_ROWS 4u  /* rows of dX without an adapter get their base row    */

/*
 * moegg_lora_fwd -- low-rank adapters of many requests at once, added to a
 * shared projection's output: for sorted position p of adapter a and row
 * i = gather_idx[p],
 *   h[p, r] = sum_k X[i, k] * A[a, r, k]                      r < ranks[a]
 *   Y[i, n] = base[i, n] + scales[a] * sum_r h[p, r] * B[a, n, r]
 * The rows are grouped by moegg_route over one adapter id a row (topk 1), once
 * for all projections of a batch.  With m_sizes and rows in expert order
 * (gather_idx NULL) the same call adapts the experts' products, L = E.
 *
 *   X          rows of K elements of `dtype` (MOEGG_BF16 or MOEGG_FP16), ldx
 *              elements apart.
 *   A, B       [L, R, K] and [L, N, R] of `dtype`, contiguous.
 *   m_sizes    [L] int32 rows of each adapter (0 allowed).
 *   gather_idx [T] int32: row at sorted position p; entries are distinct.
 *              NULL: i = p.  An entry outside [0, T) raises
 *              MOEGG_DERR_GATHER and is skipped.
 *   ranks      [L] int32 in [0, R], or NULL for R everywhere.  Rows of A and
 *              columns of B at or past an adapter's rank are not read into the
 *              result; rank 0 is no adapter (Y = base).
 *   scales     [L] fp32, or NULL for 1.
 *   base, Y    rows of N elements, ld_base and ldy apart.  base NULL: Y holds
 *              the projection's output and is added to in place (base = Y
 *              says the same).  They overlap in no other way.
 *   H          out [T, R] fp32: h by sorted position, columns at or past the
 *              rank zero, for the backward; or NULL.
 *   workspace  device, 16-byte aligned, moegg_lora_workspace_bytes(...) bytes,
 *              no initialisation.
 * Rows at no sorted position below the sum of m_sizes (moegg_route's dropped
 * ids) keep what Y holds; moegg_lora_fwd_all_rows gives them their base row.
 * H's rows at positions from that sum on are left as they were.  h is kept in
 * fp32 and enters the second product with all 24 bits of its mantissa in bf16
 * and 22 in fp16; sums in fp32; Y is rounded once.
 * Bit-for-bit deterministic.  Any K and N from 8 on and any strides; rows need
 * the alignment of one element.  T = 0 is a no-op.
 * Errors: ESHAPE for T < 0, L outside [1, MOEGG_MAX_EXPERTS], R outside
 * [1, MOEGG_MAX_LORA_RANK], K or N < 8, a row stride below its row or past
 * 2^31, sizes past 2^40 bytes or past what a launch holds (2^27 rows); EUNSUPPORTED for MOEGG_FP32; EINVAL for an unknown dtype, NULL
 * or misaligned pointers, base = Y with different strides; EWORKSPACE.
 */
moegg_status moegg_lora_fwd(const void *X, int64_t ldx, const void *A, const void *B,
                            const int32_t *m_sizes, const int32_t *gather_idx,
                            const int32_t *ranks, const float *scales, int32_t dtype,
                            int64_t num_rows, int32_t num_adapters, int32_t R, int32_t K,
                            int32_t N, const void *base, int64_t ld_base, void *Y, int64_t ldy,
                            float *H, void *workspace, size_t workspace_bytes,
                            int32_t *error_flags, void *stream);

/*
 * moegg_lora_fwd that writes every row of Y: a row without an adapter gets its
 * base row, Y[i] = base[i].  For a Y apart from base that holds nothing yet;
 * with base NULL or Y itself the two calls are the same.
 */
moegg_status moegg_lora_fwd_all_rows(const void *X, int64_t ldx, const void *A, const void *B, const
                                     int32_t *m_sizes, const int32_t *gather_idx, const int32_t
                                     *ranks, const float *scales, int32_t dtype, int64_t num_rows,
                                     int32_t num_adapters, int32_t R, int32_t K, int32_t N, const
                                     void *base, int64_t ld_base, void *Y, int64_t ldy, float *H,
                                     void *workspace, size_t workspace_bytes, int32_t *error_flags,
                                     void *stream);

/* Workspace of moegg_lora_fwd; 0 for sizes it refuses. */
size_t moegg_lora_workspace_bytes(int64_t num_rows, int32_t num_adapters, int32_t R, int32_t K,
                                  int32_t N);

/*
 * moegg_lora_bwd -- gradients of moegg_lora_fwd:
 *   dh[p, r]    = scales[a] * sum_n dY[i, n] * B[a, n, r]     r < ranks[a]
 *   dX[i, k]    = base[i, k] + sum_r dh[p, r] * A[a, r, k]
 *   dA[a, r, k] = sum_{p of a} dh[p, r] * X[i, k]
 *   dB[a, n, r] = scales[a] * sum_{p of a} dY[i, n] * H[p, r]
 *   H          the forward's H.
 *   base, dX   as base and Y in the forward (base: the shared projection's
 *              input gradient; rows without an adapter keep what dX holds, or
 *              get their base row with LORA_ALL_ROWS); dX NULL skips it.  dX
 *              may not overlap X or dY when dA and dB are asked for (EINVAL):
 *              both are read after dX is written.
 *   dA, dB     out [L, R, K] and [L, N, R] of `dtype`, fp32 with
 *              MOEGG_LORA_FP32_GRAD; every element is written, zeros for
 *              adapters without rows and past an adapter's rank.  Both NULL
 *              skips them (X and H are then not read and may be NULL).
 *   workspace  moegg_lora_bwd_workspace_bytes(...) bytes.
 * dh and H enter the products as h does in the forward.
 * Arguments, determinism and errors otherwise as in the forward;
 * EINVAL for one of dA and dB without the other.  T = 0 writes zeros to dA
 * and dB.
 */
moegg_status moegg_lora_bwd(const void *X, int64_t ldx, const void *dY, int64_t lddy,
                            const void *A, const void *B, const float *H, const int32_t *m_sizes,
                            const int32_t *gather_idx, const int32_t *ranks, const float *scales,
                            int32_t dtype, int64_t num_rows, int32_t num_adapters, int32_t R,
                            int32_t K, int32_t N, const void *base, int64_t ld_base, void *dX,
                            int64_t lddx, void *dA, void *dB, uint32_t flags, void *workspace,
                            size_t workspace_bytes, int32_t *error_flags, void *stream);

/* Workspace of moegg_lora_bwd; 0 for sizes it refuses. */
size_t moegg_lora_bwd_workspace_bytes(int64_t num_rows, int32_t num_adapters, int32_t R,
                                      int32_t K, int32_t N);

/*
 * moegg_quant_rows -- rows in 8-bit integers with a scale for each row: what
 * moegg_grouped_gemm_i8 takes for its tokens and, laid out once, its weights
 * ([E * N] rows of K).
 *
 *   scales[i] = m / 127, m = max_k |X[i, k]|            (fp32)
 *   Q[i, k]   = round(127 X[i, k] / m)                  (real quotient, ties to even)
 *
 * so |Q| <= 127, and scales[i] * Q[i, k] is X[i, k] to half a scale.  A row of
 * zeros gets scale 0 and codes 0; a row that holds an infinity or NaN scale
 * NaN and codes 0.
 *   X       [rows, K] of `dtype`, rows ldx >= K elements apart.
 *   Q       out [rows, Kq], Kq = K rounded up to a multiple of 16, 16-byte
 *           aligned; columns from K on are zeros.
 *   scales  out [rows] fp32.
 * rows = 0 is a no-op.  Outputs overlap neither X nor each other.  More rows than
 * 2^24 - 1 take several calls.  Errors: ESHAPE for rows < 0 or past that, K < 1 or past
 * 2^30, ldx < K, sizes past 2^40 bytes; EINVAL for an unknown dtype, NULL or misaligned
 * pointers.
 */
moegg_status moegg_quant_rows(const void *X, int32_t dtype, int64_t ldx, int64_t rows, int32_t K,
                              int8_t *Q, float *scales, void *stream);

/*
 * moegg_grouped_gemm_i8 -- moegg_grouped_gemm_fwd on 8-bit integers: for
 * sorted position p of expert e and row i = src(p) of Xq,
 *   y[n] = x_scales[i] * w_scales[e, n] * sum_k Xq[i, k] * Wq[e, n, k]
 * The sum is exact (int32), the scales are applied in fp32.  src, the
 * permute flags and FUSE_MUL_POST as in the forward, Y bf16 rounded once.
 *   MOEGG_GATED_SILU or MOEGG_GATED_GELU: Y [S, N/2] = act(gate) * linear with
 *   act(g) = g / (1 + e^-g), or g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)));
 *   either is 0 where it is above -1.1e-36 and e^-g (e^-2y of tanh y) past 2^126;
 *   W rows in (gate, linear) pairs, or with MOEGG_GATED_HALVES the N/2 gate
 *   rows first.  Not with PERMUTE_Y or FUSE_MUL_POST.
 *
 *   Xq        [T or S, K] int8, x_scales [T or S] fp32; Wq [E, N, K] int8,
 *             w_scales [E, N] fp32: as moegg_quant_rows writes them.  K is
 *             the padded row length Kq, a multiple of 16.  Any int8 value.
 *   others    as in the forward; 2 GiB at most for Xq and for one expert's Wq.
 * Rows at positions past the sum of m_sizes are left as they were.  T = 0 is a
 * no-op.  Y overlaps no input.  Errors: as the forward, and ESHAPE for K not a multiple of 16 or past
 * MOEGG_MAX_I8_K, Xq or Wq not 16-byte aligned; EINVAL for both activations,
 * HALVES without one, or an overlap.
 */
moegg_status moegg_grouped_gemm_i8(const int8_t *Xq, const float *x_scales, const int8_t *Wq,
                                   const float *w_scales, const int32_t *m_sizes,
                                   const int32_t *gather_idx, const float *topk_weights,
                                   int32_t num_tokens, int32_t topk, int32_t num_experts,
                                   int32_t N, int32_t K, uint32_t flags, void *Y,
                                   int32_t *error_flags, void *stream);

/*
 * moegg_pack8 -- an activation kept in 8 bits until the backward pass: 8.25
 * bits a value.  Blocks of 32 neighbours of a row share a power of two,
 *   step = 2^(b - 127), the smallest with round(max |x| / step) <= 127, b >= 1
 *   code = round(x / step)                               (ties to even)
 * code * step is exact in bf16 (and fp32), so that reading it back loses
 * nothing more.  b is at most 248, where codes are held at +-127 (magnitudes past
 * 127.5 * 2^121).  A block that holds an infinity or NaN gets b = 255 and reads
 * back as NaN.
 *   X       [rows, cols] of `dtype`, rows ldx >= cols elements apart.
 *   Q       out [rows, Cp] int8, Cp = cols rounded up to a multiple of 32,
 *           16-byte aligned; codes from cols on are 0.
 *   scales  out [rows, Cp / 32], the bytes b.
 * rows = 0 is a no-op.  Outputs overlap neither X nor each other.  Errors:
 * ESHAPE for rows < 0, cols < 1 or past 2^30, ldx < cols, sizes past 2^40
 * bytes; EINVAL for an unknown dtype, NULL or misaligned pointers.
 */
moegg_status moegg_pack8(const void *X, int32_t dtype, int64_t ldx, int64_t rows, int32_t cols,
                         int8_t *Q, uint8_t *scales, void *stream);

/*
 * moegg_unpack8 -- X[i, c] = Q[i, c] * 2^(scales[i, c / 32] - 127), rounded to
 * `dtype` (fp16: held at +-65504).  Arguments and errors as moegg_pack8.
 */
moegg_status moegg_unpack8(const int8_t *Q, const uint8_t *scales, int64_t rows, int32_t cols,
                           void *X, int32_t dtype, int64_t ldx, void *stream);

/*
 * moegg_gated_fwd -- the gated feed-forward block's first half in one kernel,
 * for training: both projections, the activation and the product, and what
 * the backward needs of them.  For sorted position p of expert e
 *   A[p, :] = X[src(p), :] W_e^T       W [E, 2 I, K]: gate and linear rows
 *   H[p, c] = act(g) * u               g, u: columns c of A's gate and linear part
 * from the fp32 sums, rounded once.  Flags: PERMUTE_X as in the forward;
 * GATED_SILU or GATED_GELU (one of them), with GATED_HALVES W's and A's gate
 * part first instead of pairs.
 *
 *   X      bf16 [T, K] (PERMUTE_X) or [S, K].
 *   H      out bf16 [S, I].
 *   A      out bf16 [S, 2 I], in W's order of rows, or NULL.
 *   Aq, As out: g and u packed as by moegg_pack8 from their fp32 sums, or both
 *          NULL: Aq [S, 2 Ip] int8, the gate codes and then the linear ones,
 *          Ip = I rounded up to a multiple of 32; As [S, 2 Ip / 32].  Aq 16-byte
 *          aligned.  Not together with A.
 *   workspace  device, 16-byte aligned, moegg_gated_fwd_workspace_bytes(...)
 *          bytes: X and the used experts' W in rows of whole 16-byte chunks,
 *          needed when K is not a multiple of 8 or X or W is not 16-byte
 *          aligned; else may be NULL.  No initialisation.
 * Rows at positions past the sum of m_sizes are left as they were.  T = 0 is a
 * no-op.  Outputs and the workspace overlap no input and not each other; a
 * workspace serves one call at a time.  Errors: EINVAL for flags other than
 * these, none or both activations, Aq without As (or As without Aq, or A beside
 * them), NULL or misaligned pointers, an overlap; ESHAPE for sizes as in the forward, I < 1; EWORKSPACE.
 */
moegg_status moegg_gated_fwd(const void *X, const void *W, const int32_t *m_sizes,
                             const int32_t *gather_idx, int32_t num_tokens, int32_t topk,
                             int32_t num_experts, int32_t I, int32_t K, uint32_t flags, void *H,
                             void *A, int8_t *Aq, uint8_t *As, void *workspace,
                             size_t workspace_bytes, int32_t *error_flags, void *stream);

/* Workspace of moegg_gated_fwd for rows that are not whole 16-byte chunks (K not
 * a multiple of 8, or operands not 16-byte aligned); 0 for sizes it refuses. */
size_t moegg_gated_fwd_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts,
                                       int32_t I, int32_t K, uint32_t flags);

/*
 * moegg_gated_bwd -- from the down projection's output gradient to the gradient
 * of moegg_gated_fwd's A, in one kernel: for sorted position p of expert e
 *   dH[p, c] = sum_n dY[q(p), n] * W[e, n, c]            (fp32, not rounded)
 *   dg = dH * u * act'(g),  du = dH * act(g)             rounded once to dA
 *   H[p, c] = act(g) * u                                 when H is not NULL
 * with g and u as the forward kept them (A, or Aq and As).  H, from the kept
 * values, is the X of the down projection's dW; dA is the dY of the first
 * projections' dX and dW (moegg_grouped_gemm_dX / _dW with N = 2 I).
 *
 *   dY    bf16 [S, N]; q(p) = gather_idx[p] with PERMUTE_Y (the flag of the
 *         down projection's forward), else p.
 *   W     bf16 [E, N, I], the down projection's weight.
 *   dA    out bf16 [S, 2 I] in A's order; may be A itself.
 *   flags PERMUTE_Y, GATED_SILU or GATED_GELU, GATED_HALVES.
 *   workspace  as moegg_gated_fwd's, moegg_gated_bwd_workspace_bytes(...)
 *         bytes: needed when N or I is not a multiple of 8 or dY or W is not
 *         16-byte aligned.
 * Rows of dA and H at positions past the sum of m_sizes, and rows whose gather
 * entry is bad, are left as they were.  T = 0 is a no-op.  Overlaps and errors
 * as moegg_gated_fwd, dA over A excepted; exactly one of A and (Aq, As) is given (EINVAL).
 */
moegg_status moegg_gated_bwd(const void *dY, const void *W, const int32_t *m_sizes,
                             const int32_t *gather_idx, const void *A, const int8_t *Aq,
                             const uint8_t *As, int32_t num_tokens, int32_t topk,
                             int32_t num_experts, int32_t N, int32_t I, uint32_t flags, void *dA,
                             void *H, void *workspace, size_t workspace_bytes,
                             int32_t *error_flags, void *stream);

/* Workspace of moegg_gated_bwd for rows that are not whole 16-byte chunks; 0 for
 * sizes it refuses. */
size_t moegg_gated_bwd_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts,
                                       int32_t N, int32_t I);

/*
 * moegg_grouped_gemm_dW_packed -- moegg_grouped_gemm_dW with X as moegg_pack8
 * keeps it: Xq [T or S, Cp] int8 and x_scales [T or S, Cp / 32], Cp = K rounded up to
 * a multiple of 32.  The rows are expanded to bf16 (without loss) in the
 * workspace, in expert order where that pays, and reduced there; everything
 * else, the split of hot experts among it, as moegg_grouped_gemm_dW.
 *   workspace  device, 16-byte aligned, required:
 *              moegg_grouped_gemm_dW_packed_workspace_bytes(...) bytes.
 * dW and the workspace overlap no input and not each other (EINVAL).
 */
moegg_status moegg_grouped_gemm_dW_packed(const int8_t *Xq, const uint8_t *x_scales,
                                          const void *dY, const int32_t *m_sizes,
                                          const int32_t *gather_idx, int32_t num_tokens,
                                          int32_t topk, int32_t num_experts, int32_t N, int32_t K,
                                          uint32_t flags, void *dW, void *workspace,
                                          size_t workspace_bytes, int32_t *error_flags,
                                          void *stream);

size_t moegg_grouped_gemm_dW_packed_workspace_bytes(int32_t num_tokens, int32_t topk,
                                                    int32_t num_experts, int32_t N, int32_t K,
                                                    uint32_t flags);

#ifdef __cplusplus
}
#endif

#endif /* MOEGG_H */
