// dg_route.cuh — routing of tokens to experts: scores, group-limited top-k choice with a balance
// bias, weights, and the gradient of the logits (sm_100a).
//
// For one token with logits x[E]:
//   s = softmax(x) or sigmoid(x);  choice value c = s + bias (bias optional);
//   groups of E/groups experts are ranked by the sum of their group_top (1 or 2) largest c and
//   the topk_groups best are kept; the k largest c of the kept groups are chosen, equal values
//   in the order of their index; w_j = s[id_j], divided by the chosen scores' sum when renorm,
//   times scale.
// A logit of -inf or NaN and a bias of -inf or NaN take an expert out of the choice (NaN also
// sets the error word); +inf counts as the largest finite fp32. Places that no expert fills get
// id -1 and weight 0.
#pragma once
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "dg_norm.cuh"
#include "dg_ptx.cuh"

namespace dg {

enum : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };
constexpr int ROUTE_WARPS = 4;   // tokens per block
constexpr int ROUTE_MAX_E = 1024, ROUTE_MAX_K = 32, ROUTE_MAX_GROUPS = 32;

struct RouteParams {
    const void *logits;     // [T,E]
    const float *bias;      // [E] or NULL
    int32_t *ids;           // [T,k]
    float *weights;         // [T,k]
    const float *grad_w;    // backward: [T,k]
    void *grad_logits;      // backward: [T,E]
    int *err;
    int T, E, k, groups, topk_groups, group_top, score, renorm;
    float scale;
};

__device__ __forceinline__ float route_logit(float x, int *err) {
    if (x != x) {
        report_error(err, ERR_DATA);
        return -CUDART_INF_F;
    }
    return fminf(x, CUDART_MAX_NORMAL_F);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// sigmoid(x)·exp(-m), m = min(largest x of the row, 0): an x >= 0 comes with m = 0 only.
__device__ __forceinline__ float sigmoid_scaled(float x, float m) {
    return x >= 0.f ? 1.f / (1.f + expf(-x)) : expf(x - m) / (1.f + expf(x));
}

__device__ __forceinline__ double sigmoid_f64(double x) {
    if (x >= 0.0) return 1.0 / (1.0 + exp(-x));
    const double e = exp(x);
    return e / (1.0 + e);
}

// Weights of the chosen logits, one per lane (`in`: the lane holds one). `row_max`, `row_sum`: of
// exp(x - row_max) over the row's logits, for softmax without renorm. With renorm the scores
// are taken relative to the largest chosen one, so that no sum of them is zero.
__device__ __forceinline__ float route_weight(const RouteParams &p, float scale, bool in, float x, float row_max,
                                              float row_sum) {
    if (!p.renorm) {
        if (!in) return 0.f;
        return scale * (p.score == SCORE_SOFTMAX ? expf(x - row_max) / row_sum : sigmoid_scaled(x, 0.f));
    }
    const float m = warp_max(in ? x : -CUDART_INF_F);
    float s = 0.f;
    if (in) s = p.score == SCORE_SOFTMAX ? expf(x - m) : sigmoid_scaled(x, fminf(m, 0.f));
    const float sum = warp_sum(s);
    return in ? scale * (s / sum) : 0.f;
}

// A warp per token; lane l holds the experts l, l + 32, ... (EPL of them) in registers.
// Values that decide the choice are 64-bit: two scores that differ by less than an fp32 rounding
// keep the order of their real values.
template <typename LT, int EPL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_kernel(const RouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const LT *row = static_cast<const LT *>(p.logits) + static_cast<size_t>(t) * p.E;
    float x[EPL];
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        x[i] = e < p.E ? route_logit(static_cast<float>(row[e]), p.err) : -CUDART_INF_F;
        mx = fmaxf(mx, x[i]);
    }
    const bool softmax = p.score == SCORE_SOFTMAX;
    float sum = 0.f;
    double sum64 = 0.0;
    if (softmax) {
        mx = warp_max(mx);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (x[i] > -CUDART_INF_F) sum += expf(x[i] - mx);
        sum = warp_sum(sum);
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (x[i] > -CUDART_INF_F) sum64 += exp(static_cast<double>(x[i]) - static_cast<double>(mx));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum64 += __shfl_xor_sync(0xFFFFFFFFu, sum64, o);
        }
    }
    // choice values: the score plus the bias; without a bias the logit itself, which is in the
    // same order as its score
    double c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        c[i] = x[i];
        if (p.bias && x[i] > -CUDART_INF_F) {
            const float b = p.bias[e];
            if (b != b) report_error(p.err, ERR_DATA);
            const double s = softmax ? exp(static_cast<double>(x[i]) - static_cast<double>(mx)) / sum64
                                     : sigmoid_f64(static_cast<double>(x[i]));
            c[i] = b > -CUDART_INF_F ? s + static_cast<double>(b) : -CUDART_INF;
        }
    }
    if (p.groups > 1) {
        const int gs = p.E / p.groups;
        double mine = -CUDART_INF;   // lane g: the value of group g
        for (int g = 0; g < p.groups; ++g) {
            double a = -CUDART_INF, b = -CUDART_INF;   // the two largest
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * 32 + lane;
                if (e >= g * gs && e < (g + 1) * gs) {
                    b = fmax(b, fmin(a, c[i]));
                    a = fmax(a, c[i]);
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const double a2 = __shfl_xor_sync(0xFFFFFFFFu, a, o), b2 = __shfl_xor_sync(0xFFFFFFFFu, b, o);
                b = fmax(fmin(a, a2), fmax(b, b2));
                a = fmax(a, a2);
            }
            double v = a;
            if (p.group_top == 2 && a > -CUDART_INF) {
                if (!p.bias) {   // back from logits to scores (softmax: times the row's sum)
                    a = softmax ? exp(a - static_cast<double>(mx)) : sigmoid_f64(a);
                    if (b > -CUDART_INF) b = softmax ? exp(b - static_cast<double>(mx)) : sigmoid_f64(b);
                }
                v = b > -CUDART_INF ? a + b : a;
            }
            if (lane == g) mine = v;
        }
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const double v = __shfl_sync(0xFFFFFFFFu, mine, h);
            rank += (v > mine || (v == mine && h < lane)) ? 1 : 0;
        }
        const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < p.groups && rank < p.topk_groups);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane;
            if (e < p.E && !((kept >> (e / gs)) & 1u)) c[i] = -CUDART_INF;
        }
    }
    int my_id = -1;
    float my_x = 0.f;
    for (int j = 0; j < p.k; ++j) {
        double best = -CUDART_INF;
        int e = -1;
        float xe = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (c[i] > best) {
                best = c[i];
                e = i * 32 + lane;
                xe = x[i];
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const double b2 = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            const int e2 = __shfl_xor_sync(0xFFFFFFFFu, e, o);
            const float x2 = __shfl_xor_sync(0xFFFFFFFFu, xe, o);
            if (b2 > best || (b2 == best && e2 < e)) {
                best = b2;
                e = e2;
                xe = x2;
            }
        }
        if (best == -CUDART_INF) break;   // the same in every lane
        if (lane == j) {
            my_id = e;
            my_x = xe;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i * 32 + lane == e) c[i] = -CUDART_INF;
    }
    const float w = route_weight(p, p.scale, my_id >= 0, my_x, mx, sum);
    if (lane < p.k) {
        p.ids[static_cast<size_t>(t) * p.k + lane] = my_id;
        p.weights[static_cast<size_t>(t) * p.k + lane] = w;
    }
}

// Gradient of the logits from the gradient g of the weights; a warp per token, lane j the
// choice j (id -1: none). With o_j = s_j / (the chosen scores' sum):
//   softmax, renorm:  dx_j = scale·o_j·(g_j - sum_i g_i·o_i), the other logits cancel out;
//   sigmoid, renorm:  the same times (1 - s_j);
//   sigmoid:          dx_j = scale·g_j·s_j·(1 - s_j);
//   softmax:          dx_e = s_e·(scale·g_e - sum_i scale·g_i·s_i) for every e (g_e = 0 unless chosen).
// A choice that stands twice in a row adds both gradients.
template <typename LT>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_backward_kernel(const RouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const LT *row = static_cast<const LT *>(p.logits) + static_cast<size_t>(t) * p.E;
    LT *out = static_cast<LT *>(p.grad_logits) + static_cast<size_t>(t) * p.E;
    int id = -1;
    float g = 0.f, x = 0.f;
    if (lane < p.k) {
        id = p.ids[static_cast<size_t>(t) * p.k + lane];
        if (id >= p.E) {
            report_error(p.err, ERR_DATA);
            id = -1;
        }
        if (id >= 0) {
            g = p.grad_w[static_cast<size_t>(t) * p.k + lane];
            x = fminf(static_cast<float>(row[id]), CUDART_MAX_NORMAL_F);
        }
    }
    const bool in = id >= 0, full = p.score == SCORE_SOFTMAX && !p.renorm;
    float mx = -CUDART_INF_F, sum = 0.f;
    if (full) {
        for (int e = lane; e < p.E; e += 32) mx = fmaxf(mx, route_logit(static_cast<float>(row[e]), nullptr));
        mx = warp_max(mx);
        for (int e = lane; e < p.E; e += 32) {
            const float v = route_logit(static_cast<float>(row[e]), nullptr);
            if (v > -CUDART_INF_F) sum += expf(v - mx);
        }
        sum = warp_sum(sum);
    }
    const float o = route_weight(p, 1.f, in, x, mx, sum);   // o_j or s_j
    const float total = warp_sum(in ? g * o : 0.f);
    float dx = in ? p.scale * (o * (p.renorm ? g - total : g)) : 0.f;
    if (in && p.score == SCORE_SIGMOID) dx *= sigmoid_scaled(-x, 0.f);
    for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        float v = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const int idj = __shfl_sync(0xFFFFFFFFu, id, j);
            const float dj = __shfl_sync(0xFFFFFFFFu, dx, j);
            if (idj == e) v += dj;
        }
        if (e < p.E) {
            if (full) {
                const float xe = route_logit(static_cast<float>(row[e]), nullptr);
                if (xe > -CUDART_INF_F) v -= p.scale * (total * (expf(xe - mx) / sum));
            }
            store_vec<LT, 1>(out + e, &v);
        }
    }
}

}  // namespace dg
