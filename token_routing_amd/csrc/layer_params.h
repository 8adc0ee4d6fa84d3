// Kernel parameter blocks and host launchers of the operators around the
// grouped GEMMs: the gate and the sort of token rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moegg {

// Gate: ids and weights of each token's top-k experts from its logits.
struct GateParams {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    float *scores;
    int32_t *err;
    int64_t T, ld;
    int E, topk, n_groups, topk_groups;
    int dtype;
    float scale;
    bool sigmoid, renorm;
};

struct GateBwdParams {
    const void *logits;
    const int32_t *ids;
    const float *dweights;
    const float *dscores;
    void *dlogits;
    int32_t *err;
    int64_t T, ld;
    int E, topk;
    int dtype;
    float scale;
    bool sigmoid, renorm;
};

// Token rows out to expert-ordered rows: dst[row(s)] = w[s] * src[t], and,
// with dw, dw[s] = <src[t], other[row(s)]>.  padded != null: `map` is the
// unpadded order, row() adds each expert's padding, row_map receives it, and
// pad rows are cleared.
struct SpreadParams {
    const void *src;
    const void *other;
    const int32_t *map;
    const float *weights;
    const int32_t *offsets;
    const int32_t *padded;
    void *dst;
    int32_t *row_map;
    float *dw;
    int32_t *err;
    int64_t T, rows;
    int topk, E, K;
    bool map_is_padded;
    int pad_blocks;  // workgroups per expert that clear pad rows
};

// Expert-ordered rows back to token rows: out[t] = base[t] + sum_j w[s] *
// rows_in[row(s)], and, with dw, dw[s] = <other[t], rows_in[row(s)]>.
struct CollectParams {
    const void *rows_in;
    const void *base;
    const void *other;
    const int32_t *map;
    const float *weights;
    void *out;
    float *dw;
    int32_t *err;
    int64_t T, rows;
    int topk, K;
};

hipError_t gate_launch(const GateParams &p, hipStream_t stream);
hipError_t gate_bwd_launch(const GateBwdParams &p, hipStream_t stream);
hipError_t spread_launch(const SpreadParams &p, int dtype, hipStream_t stream);
hipError_t collect_launch(const CollectParams &p, int dtype, hipStream_t stream);

}  // namespace moegg
