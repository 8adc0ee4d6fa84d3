// The gate: from a token's E router logits to the ids and weights of its
// top-k experts, and the gradient of the logits, gfx950.
//
//   score_i = softmax(l)_i  or  1 / (1 + exp(-l_i))
//   key_i   = score_i + bias_i, the k largest picked (ties: lowest index),
//             with groups only inside the topk_groups groups of largest
//             value, a group's value being the sum of its two largest keys
//   w_j     = scale * score_{id_j}  (renorm: / sum over the picked scores)
//
// A token is held by G = 8 to 64 lanes of one wave, V logits a lane, all in
// registers: the logits are read once, and maxima, sums and the k picks are
// reductions over the G lanes, which bound the kernel (its bytes would take a
// fifth of the time, a fifteenth with keys in 64 bits).  Both scores rise with the logit, so without
// bias and groups the picks compare the logits themselves and need no exp;
// with them the keys are computed and compared in 64 bits, because keys of
// different experts come as close as a rounding of 32 bits and the pick must
// not depend on it.  With renorm the weights of a softmax are the softmax
// over the picked logits (of a sigmoid, over their log-sigmoids): no sum that
// can underflow is divided by.
//
// Backward, with q_j = w_j / scale and g the weights' gradient:
//   renorm:  dl_{id_j} = scale * q_j * (g_j - sum_m q_m g_m)   [softmax]
//            the same times (1 - score_{id_j})                 [sigmoid]
//   plain:   ds_{id_j} += scale * g_j, then through the score:
//            dl_i = p_i (ds_i - sum ds p)  or  ds_i s_i (1 - s_i)
#include "elems.h"

#include "layer_params.h"

namespace moegg {

namespace {

constexpr int kGateThreads = 256;
constexpr int kErrLogit = 8;  // MOEGG_DERR_LOGIT
constexpr float kNegInf = -__builtin_huge_valf();

// Every lane of a group of G combined with op (commutative), all lanes ending
// with the result: moves inside the registers (quad and mirror moves up to 16
// lanes, row and half exchanges above).  The same through LDS shifts took four
// fifths of a call's time.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true);
}
template <int G, class Op> __device__ __forceinline__ uint32_t lanes_combine(uint32_t v, Op op)
{
    v = op(v, dpp<0xb1>(v));   // quad_perm [1,0,3,2]
    v = op(v, dpp<0x4e>(v));   // quad_perm [2,3,0,1]
    v = op(v, dpp<0x141>(v));  // row_half_mirror
    if constexpr (G >= 16)
        v = op(v, dpp<0x140>(v));  // row_mirror
    if constexpr (G >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    if constexpr (G >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    return v;
}
template <int G> __device__ __forceinline__ uint32_t lanes_umax(uint32_t v)
{
    return lanes_combine<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G> __device__ __forceinline__ uint32_t lanes_umin(uint32_t v)
{
    return lanes_combine<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G> __device__ __forceinline__ float lanes_max(float v)
{
    return __builtin_bit_cast(
        float, lanes_combine<G>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
            return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a),
                                                      __builtin_bit_cast(float, b)));
        }));
}
template <int G> __device__ __forceinline__ float lanes_sum(float v)
{
    return __builtin_bit_cast(
        float, lanes_combine<G>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) +
                                                    __builtin_bit_cast(float, b));
        }));
}
template <int G> __device__ __forceinline__ double lanes_sum(double v)
{
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1)
        v += __shfl_xor(v, d, kWave);
    return v;
}

// Order-preserving bits: a < b as floats iff bits(a) < bits(b); every finite
// value maps above 0, which stands for an expert that cannot be picked.
__device__ __forceinline__ uint32_t order_bits(float f)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 becomes +0
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits(uint32_t u)
{
    return __builtin_bit_cast(float, (u >> 31) ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t order_bits(double f)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, f + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ float sigmoid_of(float l)
{
    return 1.0f / (1.0f + expf(-l));
}
__device__ __forceinline__ float log_sigmoid_of(float l)
{
    return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}

// The lane's V logits of experts [lane * V, lane * V + V) of one row;
// experts at or past E, and rows that are not live, read as -inf.
template <int V, int DT>
__device__ __forceinline__ void load_row(float (&l)[V], const void *logits, int64_t row, int lane,
                                         int E, bool live)
{
    typedef typename Elem<DT>::store_t st_t;
    typedef st_t vec_t __attribute__((ext_vector_type(V), aligned(sizeof(st_t))));
    const st_t *p = static_cast<const st_t *>(logits) + row + lane * V;
    if (live && lane * V + V <= E) {
        if constexpr (V == 1) {
            l[0] = Elem<DT>::widen(p[0]);
        } else {
            const vec_t v = *reinterpret_cast<const vec_t *>(p);
#pragma unroll
            for (int i = 0; i < V; ++i)
                l[i] = Elem<DT>::widen(v[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        l[i] = (live && lane * V + i < E) ? Elem<DT>::widen(p[i]) : kNegInf;
}

template <int V>
__device__ __forceinline__ void load_row(float (&l)[V], const void *logits, int dtype, int64_t row,
                                         int lane, int E, bool live)
{
    if (dtype == kBf16)
        load_row<V, kBf16>(l, logits, row, lane, E, live);
    else if (dtype == kFp16)
        load_row<V, kFp16>(l, logits, row, lane, E, live);
    else
        load_row<V, kFp32>(l, logits, row, lane, E, live);
}

__device__ __forceinline__ float load_one(const void *logits, int dtype, int64_t at)
{
    return dtype == kBf16   ? Elem<kBf16>::widen(static_cast<const uint16_t *>(logits)[at])
           : dtype == kFp16 ? Elem<kFp16>::widen(static_cast<const uint16_t *>(logits)[at])
                            : static_cast<const float *>(logits)[at];
}

template <int V>
__device__ __forceinline__ void store_row_f32(float *p, const float (&f)[V], int lane, int E)
{
    typedef float vec_t __attribute__((ext_vector_type(V), aligned(4)));
    if (lane * V + V <= E) {
        if constexpr (V == 1) {
            p[lane] = f[0];
        } else {
            vec_t v;
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = f[i];
            *reinterpret_cast<vec_t *>(p + lane * V) = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane * V + i < E)
            p[lane * V + i] = f[i];
}

template <int V, int DT>
__device__ __forceinline__ void store_row(void *out, const float (&f)[V], int64_t row, int lane,
                                          int E)
{
    typedef typename Elem<DT>::store_t st_t;
    typedef st_t vec_t __attribute__((ext_vector_type(V), aligned(sizeof(st_t))));
    st_t *p = static_cast<st_t *>(out) + row + lane * V;
    if (lane * V + V <= E) {
        if constexpr (V == 1) {
            p[0] = Elem<DT>::narrow(f[0]);
        } else {
            vec_t v;
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = Elem<DT>::narrow(f[i]);
            *reinterpret_cast<vec_t *>(p) = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane * V + i < E)
            p[i] = Elem<DT>::narrow(f[i]);
}

// Masks what is no finite logit (l becomes -inf); true if one was NaN or +inf.
template <int V> __device__ __forceinline__ bool mask_row(float (&l)[V])
{
    bool bad = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool odd = !(l[v] < __builtin_huge_valf());
        bad |= odd;
        l[v] = odd ? kNegInf : l[v];
    }
    return bad;
}

// WIDE: keys in 64 bits (bias or groups).  The token's keys are then also in
// LDS, where one lane a group finds the group's value.
template <int G, int V, bool WIDE>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateParams a)
{
    constexpr int kTokens = kGateThreads / G;
    constexpr int kSlots = V == 1 ? 1 : 64 / G;  // picks a lane can hold
    // One more place a group, so that the groups' scans start on different banks.
    constexpr int kKeys = G * V + 64;
    __shared__ double s_key[WIDE ? kTokens * kKeys : 1];
    __shared__ double s_group[WIDE ? kTokens * 64 : 1];
    __shared__ int s_keep[WIDE ? kTokens * 64 : 1];
    const int lane = threadIdx.x % G;
    const int slot = threadIdx.x / G;
    const int64_t t = (int64_t)blockIdx.x * kTokens + slot;
    const bool live = t < a.T;

    float l[V];
    load_row<V>(l, a.logits, a.dtype, t * a.ld, lane, a.E, live);
    bool bad = mask_row<V>(l);

    float m = kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v)
        m = fmaxf(m, l[v]);
    m = lanes_max<G>(m);
    const float m0 = m > kNegInf ? m : 0.0f;  // a row without any expert

    // Scores in 32 bits: asked for, or (softmax without renorm) the weights' divisor.
    float sum = 1.0f;
    if (a.scores || (!a.sigmoid && !a.renorm)) {
        float p[V];
        if (a.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                p[v] = sigmoid_of(l[v]);
        } else {
            float part = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = expf(l[v] - m0);
                part += p[v];
            }
            part = lanes_sum<G>(part);
            sum = part > 0.0f ? part : 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                p[v] /= sum;
        }
        if (a.scores && live)
            store_row_f32<V>(a.scores + t * a.E, p, lane, a.E);
    }

    // Keys as order bits; 0 cannot be picked.  Without WIDE they are the
    // logits' and fit the high word.
    uint32_t key[V], low[WIDE ? V : 1];
    if constexpr (!WIDE) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = l[v] > kNegInf ? order_bits(l[v]) : 0;
    } else {
        double d[V], dsum = 1.0;
        if (a.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                d[v] = 1.0 / (1.0 + exp(-(double)l[v]));
        } else {
            double part = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[v] = exp((double)l[v] - (double)m0);
                part += d[v];
            }
            part = lanes_sum<G>(part);
            dsum = part > 0.0 ? part : 1.0;
        }
        double *const my = s_key + slot * kKeys;
        const int per = a.E / a.n_groups;
        const int g0 = lane * V / per, at0 = lane * V - g0 * per;
        int g = g0, at = at0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            bool ok = l[v] > kNegInf;
            if (!a.sigmoid)
                d[v] /= dsum;
            if (a.bias && e < a.E) {
                const float b = a.bias[e];
                bad |= !(b < __builtin_huge_valf());
                ok &= fabsf(b) < __builtin_huge_valf();
                d[v] += (double)b;
            }
            const uint64_t bits = ok ? order_bits(d[v]) : 0;
            key[v] = (uint32_t)(bits >> 32);
            low[v] = (uint32_t)bits;
            if (e < a.E)
                my[e + g] = ok ? d[v] : -__builtin_huge_val();
            if (++at == per) {
                at = 0;
                ++g;
            }
        }
        if (a.n_groups > 1) {
            double *const val = s_group + slot * 64;
            int *const keep = s_keep + slot * 64;
            __syncthreads();
            for (int g = lane; g < a.n_groups; g += G) {
                double first = -__builtin_huge_val(), second = first;
                for (int i = 0; i < per; i += 4) {
                    double x[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        x[u] = i + u < per ? my[g * (per + 1) + i + u] : -__builtin_huge_val();
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        second = fmax(second, fmin(first, x[u]));
                        first = fmax(first, x[u]);
                    }
                }
                val[g] = second > -__builtin_huge_val() ? first + second : first;
            }
            __syncthreads();
            for (int g = lane; g < a.n_groups; g += G) {
                const double mine = val[g];
                int ahead = 0;  // groups that come before this one
                for (int h = 0; h < a.n_groups; ++h)
                    ahead += val[h] > mine || (val[h] == mine && h < g);
                keep[g] = ahead < a.topk_groups;
            }
            __syncthreads();
            g = g0;
            at = at0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (lane * V + v < a.E && !keep[g])
                    key[v] = 0;
                if (++at == per) {
                    at = 0;
                    ++g;
                }
            }
        }
    }
    if (bad && live)
        raise_error(a.err, kErrLogit);

    int pick_id[kSlots];
    float pick_l[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        pick_id[s] = -1;
        pick_l[s] = kNegInf;
    }
    for (int j = 0; j < a.topk; ++j) {
        // The largest key, then the lowest index among those that have it.
        uint32_t best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            best = key[v] > best ? key[v] : best;
        best = lanes_umax<G>(best);
        uint32_t best_low = 0;
        if constexpr (WIDE) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                best_low = key[v] == best && low[v] > best_low ? low[v] : best_low;
            best_low = lanes_umax<G>(best_low);
        }
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            if (key[v] == best && (!WIDE || low[WIDE ? v : 0] == best_low))
                at = lane * V + v;
        at = lanes_umin<G>(at);
        const int id = best ? (int)at : -1;
        const float lv = !WIDE && best ? from_order_bits(best) : kNegInf;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v == id)
                key[v] = 0;
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (j == s * G + lane) {
                pick_id[s] = id;
                pick_l[s] = lv;
            }
    }

    if constexpr (WIDE) {
        // The picks' logits again, each by the lane that holds the pick.
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (pick_id[s] >= 0 && live)
                pick_l[s] = load_one(a.logits, a.dtype, t * a.ld + pick_id[s]);
    }

    float w[kSlots];
    if (a.renorm) {
        float x[kSlots], top = kNegInf, part = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            x[s] = pick_id[s] < 0 ? kNegInf : a.sigmoid ? log_sigmoid_of(pick_l[s]) : pick_l[s];
            top = fmaxf(top, x[s]);
        }
        top = lanes_max<G>(top);
        top = top > kNegInf ? top : 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            w[s] = expf(x[s] - top);
            part += w[s];
        }
        part = lanes_sum<G>(part);
        part = part > 0.0f ? part : 1.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            w[s] /= part;
    } else {
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            w[s] = pick_id[s] < 0 ? 0.0f
                   : a.sigmoid    ? sigmoid_of(pick_l[s])
                                  : expf(pick_l[s] - m0) / sum;
    }
    if (!live)
        return;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        const int j = s * G + lane;
        if (j < a.topk) {
            a.ids[t * a.topk + j] = pick_id[s];
            a.weights[t * a.topk + j] = w[s] * a.scale;
        }
    }
}

template <int G, int V>
__global__ __launch_bounds__(kGateThreads) void gate_bwd_kernel(GateBwdParams a)
{
    constexpr int kTokens = kGateThreads / G;
    constexpr int kSlots = V == 1 ? 1 : 64 / G;
    const int lane = threadIdx.x % G;
    const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / G;
    const bool live = t < a.T;

    float l[V];
    load_row<V>(l, a.logits, a.dtype, t * a.ld, lane, a.E, live);
    mask_row<V>(l);
    float dl[V], ds[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        dl[v] = 0.0f;

    // The picks: expert, weight gradient and logit, one a lane and slot.
    int id[kSlots];
    float g[kSlots], x[kSlots];
    bool bad = false;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        const int j = s * G + lane;
        id[s] = -1;
        g[s] = 0.0f;
        x[s] = kNegInf;
        if (live && j < a.topk) {
            const int i = a.ids[t * a.topk + j];
            bad |= i >= a.E;
            if (i >= 0 && i < a.E) {
                const float one = load_one(a.logits, a.dtype, t * a.ld + i);
                if (fabsf(one) < __builtin_huge_valf()) {
                    id[s] = i;
                    x[s] = one;
                    g[s] = a.dweights[t * a.topk + j] * a.scale;
                }
            }
        }
    }
    if (bad)
        raise_error(a.err, kErrExpertId);

    float into[kSlots];  // what pick j adds to its expert: dl (renorm) or ds (plain)
    if (a.renorm) {
        float q[kSlots], y[kSlots], top = kNegInf, part = 0.0f, dot = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            y[s] = id[s] < 0 ? kNegInf : a.sigmoid ? log_sigmoid_of(x[s]) : x[s];
            top = fmaxf(top, y[s]);
        }
        top = lanes_max<G>(top);
        top = top > kNegInf ? top : 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            q[s] = expf(y[s] - top);
            part += q[s];
        }
        part = lanes_sum<G>(part);
        part = part > 0.0f ? part : 1.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            q[s] /= part;
            dot += q[s] * g[s];
        }
        dot = lanes_sum<G>(dot);
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            into[s] = id[s] < 0 ? 0.0f
                                : q[s] * (g[s] - dot) * (a.sigmoid ? sigmoid_of(-x[s]) : 1.0f);
    } else {
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            into[s] = g[s];
    }

    const bool through = a.dscores || !a.renorm;  // a gradient that passes through the scores
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        ds[v] = (a.dscores && live && e < a.E) ? a.dscores[t * a.E + e] : 0.0f;
    }
    float add[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        add[v] = 0.0f;
    const int base = (threadIdx.x & (kWave - 1)) - lane;
    // Pick j's expert and share from its lane; the picks past topk hold -1.
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
        for (int j0 = 0; j0 < min(G, a.topk - s * G); j0 += 4) {
            int e[4];
            float c[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                e[u] = __shfl(id[s], base + j0 + u, kWave);
                c[u] = __shfl(into[s], base + j0 + u, kWave);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (lane * V + v == e[u])
                        add[v] += c[u];
        }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (a.renorm)
            dl[v] = add[v];
        else
            ds[v] += add[v];
    }

    if (through) {
        if (a.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (l[v] > kNegInf)
                    dl[v] += ds[v] * sigmoid_of(l[v]) * sigmoid_of(-l[v]);
        } else {
            float m = kNegInf;
#pragma unroll
            for (int v = 0; v < V; ++v)
                m = fmaxf(m, l[v]);
            m = lanes_max<G>(m);
            m = m > kNegInf ? m : 0.0f;
            float p[V], part = 0.0f, dot = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = expf(l[v] - m);
                part += p[v];
            }
            part = lanes_sum<G>(part);
            part = part > 0.0f ? part : 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] /= part;
                dot += l[v] > kNegInf ? p[v] * ds[v] : 0.0f;
            }
            dot = lanes_sum<G>(dot);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (l[v] > kNegInf)
                    dl[v] += p[v] * (ds[v] - dot);
        }
    }
    if (!live)
        return;
    if (a.dtype == kBf16)
        store_row<V, kBf16>(a.dlogits, dl, t * a.E, lane, a.E);
    else if (a.dtype == kFp16)
        store_row<V, kFp16>(a.dlogits, dl, t * a.E, lane, a.E);
    else
        store_row<V, kFp32>(a.dlogits, dl, t * a.E, lane, a.E);
}

template <int G, int V> hipError_t gate_go(const GateParams &p, hipStream_t stream)
{
    constexpr int kTokens = kGateThreads / G;
    const dim3 grid((unsigned)((p.T + kTokens - 1) / kTokens));
    if (p.bias || p.n_groups > 1)
        hipLaunchKernelGGL((gate_kernel<G, V, true>), grid, dim3(kGateThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((gate_kernel<G, V, false>), grid, dim3(kGateThreads), 0, stream, p);
    return hipGetLastError();
}

template <int G, int V> hipError_t gate_bwd_go(const GateBwdParams &p, hipStream_t stream)
{
    constexpr int kTokens = kGateThreads / G;
    const dim3 grid((unsigned)((p.T + kTokens - 1) / kTokens));
    hipLaunchKernelGGL((gate_bwd_kernel<G, V>), grid, dim3(kGateThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t gate_launch(const GateParams &p, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    if (p.E <= 8)
        return gate_go<8, 1>(p, stream);
    if (p.E <= 64)
        return gate_go<16, 4>(p, stream);
    if (p.E <= 128)
        return gate_go<16, 8>(p, stream);
    if (p.E <= 256)
        return gate_go<32, 8>(p, stream);
    if (p.E <= 512)
        return gate_go<64, 8>(p, stream);
    return gate_go<64, 16>(p, stream);
}

hipError_t gate_bwd_launch(const GateBwdParams &p, hipStream_t stream)
{
    if (p.T == 0)
        return hipSuccess;
    if (p.E <= 8)
        return gate_bwd_go<8, 1>(p, stream);
    if (p.E <= 64)
        return gate_bwd_go<16, 4>(p, stream);
    if (p.E <= 128)
        return gate_bwd_go<16, 8>(p, stream);
    if (p.E <= 256)
        return gate_bwd_go<32, 8>(p, stream);
    if (p.E <= 512)
        return gate_bwd_go<64, 8>(p, stream);
    return gate_bwd_go<64, 16>(p, stream);
}

}  // namespace moegg
