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
constexpr int ROUTE_WARPS = 4;    // tokens per block
constexpr int ROUTE_BLOCKS = 7;   // blocks per SM (for up to 256 experts; measured with 256, below)
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
    int group_size, rows_per_group;   // E / groups; the same over 32, or 0 if that is not whole
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

// The score of a logit in 64 bits (softmax: from the row's largest logit and sum).
__device__ __noinline__ double route_score_f64(double x, double mx, double sum, bool softmax) {
    const double e = exp(softmax ? x - mx : -fabs(x));   // sigmoid: of -|x|, so that nothing overflows
    return (softmax || x < 0.0 ? e : 1.0) / (softmax ? sum : 1.0 + e);
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

// 64-bit values as integers in the same order; 0 stands for "out of the choice" (-inf).
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));   // -0 and 0 are the same
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value(uint64_t k) {
    if (k == 0) return -CUDART_INF;
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo =
        __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// The 64-bit choice value of expert e with logit x (0: out of the choice).
template <typename LT>
__device__ __forceinline__ uint64_t route_key_f64(const RouteParams &p, const LT *row, int e, float mx, double sum) {
    const float x = route_logit(static_cast<float>(row[e]), nullptr);
    if (!(x > -CUDART_INF_F)) return 0;
    if (!p.bias) return order_key(static_cast<double>(x));
    const float b = p.bias[e];
    if (!(b > -CUDART_INF_F)) return 0;
    return order_key(route_score_f64(x, mx, sum, p.score == SCORE_SOFTMAX) + static_cast<double>(b));
}

// The row's largest logit and its 64-bit sum of exp(x - largest), for softmax.
template <typename LT>
__device__ __noinline__ double route_sum_f64(const RouteParams &p, const LT *row, float mx) {
    double sum = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < p.E; e += 32) {
        const float x = route_logit(static_cast<float>(row[e]), nullptr);
        if (x > -CUDART_INF_F) sum += exp(static_cast<double>(x) - static_cast<double>(mx));
    }
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
}

// The 64-bit value of group g, the same in every lane: the sum of its group_top largest choice values.
template <typename LT>
__device__ __noinline__ double route_group_f64(const RouteParams &p, const LT *row, int g, float mx, double sum) {
    const int lane = threadIdx.x & 31;
    uint64_t a = 0, b = 0;   // the lane's two largest
#pragma unroll 1
    for (int q = lane; q < p.group_size; q += 32) {
        const uint64_t c = route_key_f64(p, row, g * p.group_size + q, mx, sum);
        b = max(b, min(a, c));
        a = max(a, c);
    }
    const uint64_t k1 = warp_max_key(a);
    const int first = __ffs(__ballot_sync(0xFFFFFFFFu, a == k1)) - 1;
    const uint64_t k2 = p.group_top == 2 ? warp_max_key(lane == first ? b : a) : 0;
    double v1 = key_value(k1), v2 = key_value(k2);
    if (!p.bias && p.group_top == 2 && k1) {   // back from logits to scores
        v1 = route_score_f64(v1, mx, sum, p.score == SCORE_SOFTMAX);
        if (k2) v2 = route_score_f64(v2, mx, sum, p.score == SCORE_SOFTMAX);
    }
    return k2 ? v1 + v2 : v1;
}

// One token by a warp with every value that decides the choice in 64 bits; lane l holds the
// experts l, l + 32, .... Taken for k > 30 and where more than 31 candidates lie too close together
// for fp32 (rows of equal fp32 logits, say). Rolled loops over a local array keep the code short: it
// is rarely in the instruction cache (unrolled or not, a token takes 12 to 14 us alone).
template <typename LT>
__device__ __noinline__ void route_token_f64(const RouteParams &p, int t) {
    const int lane = threadIdx.x & 31, n = (p.E + 31) / 32;
    const LT *row = static_cast<const LT *>(p.logits) + static_cast<size_t>(t) * p.E;
    const bool softmax = p.score == SCORE_SOFTMAX;
    uint64_t c[ROUTE_MAX_E / 32];
    float mx = -CUDART_INF_F;
    double sum = 1.0;
    if (softmax) {
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) mx = fmaxf(mx, route_logit(static_cast<float>(row[e]), nullptr));
        mx = warp_max(mx);
        sum = route_sum_f64(p, row, mx);
    }
#pragma unroll 1
    for (int i = 0; i < n; ++i) c[i] = i * 32 + lane < p.E ? route_key_f64(p, row, i * 32 + lane, mx, sum) : 0;
    if (p.groups > 1) {
        const int gs = p.group_size;
        double mine = -CUDART_INF;   // lane g: the value of group g
#pragma unroll 1
        for (int g = 0; g < p.groups; ++g) {
            const double v = route_group_f64(p, row, g, mx, sum);
            if (lane == g) mine = v;
        }
        int rank = 0;
#pragma unroll 1
        for (int h = 0; h < p.groups; ++h) {
            const double v = __shfl_sync(0xFFFFFFFFu, mine, h);
            rank += (v > mine || (v == mine && h < lane)) ? 1 : 0;
        }
        const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < p.groups && rank < p.topk_groups);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int e = i * 32 + lane;
            if (e < p.E && !((kept >> (e / gs)) & 1u)) c[i] = 0;
        }
    }
    int id = -1;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i)
            if (c[i] > best) {
                best = c[i];
                at = i;
            }
        const uint64_t m = warp_max_key(best);
        if (m == 0) break;   // the same in every lane
        const uint32_t mine = best == m ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu;
        const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, mine);
        if (mine == e) c[at] = 0;
        if (lane == j) id = static_cast<int>(e);
    }
    const float x = id >= 0 ? fminf(static_cast<float>(row[id]), CUDART_MAX_NORMAL_F) : 0.f;
    const float w = route_weight(p, p.scale, id >= 0, x, mx, static_cast<float>(sum));
    if (lane < p.k) {
        p.ids[static_cast<size_t>(t) * p.k + lane] = id;
        p.weights[static_cast<size_t>(t) * p.k + lane] = w;
    }
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid_approx(float x) { return rcp_approx(1.f + ex2_approx(-1.44269504f * x)); }

// Falling order, by a bitonic network.
template <int N>
__device__ __forceinline__ void sort_falling(float (&v)[N]) {
#pragma unroll
    for (int k = 2; k <= N; k *= 2)
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int l = i ^ j;
                if (l > i) {
                    const float hi = fmaxf(v[i], v[l]), lo = fminf(v[i], v[l]);
                    const bool falling = (i & k) == 0;
                    v[i] = falling ? hi : lo;
                    v[l] = falling ? lo : hi;
                }
            }
}

// One token by a warp; lane l holds the experts i·32 + l. True: it has to be done again in 64 bits.
//
// Choice values are fp32 from the hardware's exponential and reciprocal. The low log2(EPL) bits of a
// value are replaced by the register index i (inverted for values >= 0), so that the value names
// its expert: a lane sorts plain floats, and each choice is one maximum over the lanes' first
// values, a ballot for the lowest lane that has it, and a shift of that lane's values. Equal
// values then come in the order of their expert's index.
// Two values whose distance is within the errors (packing: EPL·2^-23 of each; sigmoid: 2^-21.5 of 1; softmax:
// 2^-18 of the largest score, from the sum) might stand in the other order, or one might be
// chosen wrongly: then all that may belong to the k largest, one in a lane, are put in the order of
// their 64-bit values, and groups at the border likewise. Neighbours with the same logit and the
// same bias are equal in truth and need no second look. With N(0,1.5) logits over 256 experts that
// is about 40 of 16384 tokens. (The softmax sum of the hardware's exponentials also divides the weights that are not
// renormalised: 2^-22 of each term and 2^-24 of its distance from the largest.)
// Bound by instructions (some 880 a token and warp with 8 groups over 256 experts): 16384 tokens take 21 us, 65536
// 71 us; every value in 64 bits took 122 us for 16384. Traffic alone would be 2.7 us. 7 blocks an SM (72 registers,
// 92 bytes of spills; 40, 20 and 4 for 128, 64 and 32 experts, where other counts were not timed) against 8, 6 and 5:
// 71, 74, 72 and 76 us for 65536 tokens. The ranking of the groups by one loop for any number of them, against one of its
// own for 8: 70.6 and 72.7 us.
template <typename LT, int EPL>
__device__ __forceinline__ bool route_token(const RouteParams &p, const float (&b)[EPL], int t, int lane) {
    const bool softmax = p.score == SCORE_SOFTMAX, by_logit = p.bias == nullptr;
    const int E = p.E, k = p.k;
    const LT *row = static_cast<const LT *>(p.logits) + static_cast<size_t>(t) * E;
    float c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        c[i] = e < E ? static_cast<float>(row[e]) : -CUDART_INF_F;
    }
    // a sum that is not finite: some logit is not, or there are fewer than 32·EPL of them
    float mx = c[0], acc = c[0], sum = 1.f;
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
        acc += c[i];
        mx = fmaxf(mx, c[i]);
    }
    const bool holes = !(fabsf(acc) <= CUDART_MAX_NORMAL_F);
    if (holes) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            bad |= c[i] != c[i];
            c[i] = c[i] == c[i] ? fminf(c[i], CUDART_MAX_NORMAL_F) : -CUDART_INF_F;
        }
        mx = c[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, c[i]);
        if (bad) report_error(p.err, ERR_DATA);
    }
    if (softmax) {
        mx = redux_max(mx);
        if (!by_logit || !p.renorm) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (c[i] > -CUDART_INF_F) sum += ex2_approx(1.44269504f * (c[i] - mx));
            sum = warp_sum(sum);
        }
    }
    const float top = softmax ? rcp_approx(sum) : 1.f;   // no score is larger
    if (!by_logit) {
        if (softmax) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                c[i] = c[i] > -CUDART_INF_F ? fmaf(top, ex2_approx(1.44269504f * (c[i] - mx)), b[i]) : -CUDART_INF_F;
        } else if (holes) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = c[i] > -CUDART_INF_F ? sigmoid_approx(c[i]) + b[i] : -CUDART_INF_F;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = sigmoid_approx(c[i]) + b[i];
        }
    }
    const float tol_score = softmax ? top * 0x1p-17f : 0x1p-20f;
    if (p.groups > 1) {
        float a1 = -CUDART_INF_F, a2 = -CUDART_INF_F;   // lane g: the two largest of group g
        if (p.rows_per_group == 1 && p.groups == EPL) {
            // A register a group: each step over the lanes halves the groups that a lane goes on with, until a lane
            // has the two largest of one group among its lanes; then lane g fetches those of group g.
            float b1[EPL], b2[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                b1[i] = c[i];
                b2[i] = -CUDART_INF_F;
            }
#pragma unroll
            for (int o = 16, m = EPL / 2; o >= 1; o >>= 1, m >>= 1) {
                const bool up = (lane & o) != 0;
                if (m >= 1) {
#pragma unroll
                    for (int h = 0; h < m; ++h) {
                        const float v1 = __shfl_xor_sync(0xFFFFFFFFu, up ? b1[h] : b1[h + m], o);
                        const float v2 = __shfl_xor_sync(0xFFFFFFFFu, up ? b2[h] : b2[h + m], o);
                        const float m1 = up ? b1[h + m] : b1[h], m2 = up ? b2[h + m] : b2[h];
                        b2[h] = fmaxf(fminf(m1, v1), fmaxf(m2, v2));
                        b1[h] = fmaxf(m1, v1);
                    }
                } else {
                    const float v1 = __shfl_xor_sync(0xFFFFFFFFu, b1[0], o), v2 = __shfl_xor_sync(0xFFFFFFFFu, b2[0], o);
                    b2[0] = fmaxf(fminf(b1[0], v1), fmaxf(b2[0], v2));
                    b1[0] = fmaxf(b1[0], v1);
                }
            }
            const int from = lane * (32 / EPL) & 31;
            a1 = __shfl_sync(0xFFFFFFFFu, b1[0], from);
            a2 = __shfl_sync(0xFFFFFFFFu, b2[0], from);
            if (lane >= EPL) a1 = a2 = -CUDART_INF_F;
        } else if (p.rows_per_group) {
            // groups of whole registers: first the two largest of each register, in lane i
            float r1 = -CUDART_INF_F, r2 = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float m1 = redux_max(c[i]);
                float m2 = m1;
                if (p.group_top == 2) {
                    const int first = __ffs(__ballot_sync(0xFFFFFFFFu, c[i] == m1)) - 1;
                    m2 = redux_max(lane == first ? -CUDART_INF_F : c[i]);
                }
                if (lane == i) {
                    r1 = m1;
                    r2 = m2;
                }
            }
            for (int q = 0; q < p.rows_per_group; ++q) {
                const int from = lane * p.rows_per_group + q;
                const float v1 = __shfl_sync(0xFFFFFFFFu, r1, from & 31), v2 = __shfl_sync(0xFFFFFFFFu, r2, from & 31);
                if (lane < p.groups) {
                    a2 = fmaxf(fminf(a1, v1), fmaxf(a2, v2));
                    a1 = fmaxf(a1, v1);
                }
            }
        } else {
            const int gs = p.group_size;
            for (int g = 0; g < p.groups; ++g) {
                float l1 = -CUDART_INF_F, l2 = -CUDART_INF_F;
                const int e0 = g * gs - lane;   // expert i·32 + lane is in the group if i·32 is in [e0, e0 + gs)
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (static_cast<unsigned>(i * 32 - e0) < static_cast<unsigned>(gs)) {
                        l2 = fmaxf(l2, fminf(l1, c[i]));
                        l1 = fmaxf(l1, c[i]);
                    }
                const float m1 = redux_max(l1);
                const int first = __ffs(__ballot_sync(0xFFFFFFFFu, l1 == m1)) - 1;
                const float m2 = redux_max(lane == first ? l2 : l1);
                if (lane == g) {
                    a1 = m1;
                    a2 = m2;
                }
            }
        }
        const bool sums = !by_logit || p.group_top == 2;   // scores, not logits, decide between the groups
        if (by_logit && sums && a1 > -CUDART_INF_F) {      // to scores (softmax: times the row's sum)
            a1 = softmax ? ex2_approx(1.44269504f * (a1 - mx)) : sigmoid_approx(a1);
            if (a2 > -CUDART_INF_F) a2 = softmax ? ex2_approx(1.44269504f * (a2 - mx)) : sigmoid_approx(a2);
        }
        // Two values are taken by halves: their sum may not fit fp32, and -inf stands for a group without experts.
        const float part = p.group_top == 2 ? 0.5f : 1.f;
        const float mine = p.group_top == 2 && a2 > -CUDART_INF_F ? part * a1 + part * a2 : part * a1;
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const float v = __shfl_sync(0xFFFFFFFFu, mine, h);
            rank += (v > mine || (v == mine && h < lane)) ? 1 : 0;
        }
        const bool keep = lane < p.groups && rank < p.topk_groups;
        uint32_t kept = __ballot_sync(0xFFFFFFFFu, keep);
        if (sums) {
            // Is the border between the groups wide enough? A group's value may be off by its scores' errors and by the
            // roundings of what was added: of both choice values, which a bias can make far larger than their sum.
            // Groups that reach across the border compete again by their 64-bit values; the others are truly above or
            // below all of those.
            const float unit = by_logit ? (softmax ? 0x1p-17f : 0x1p-20f) : tol_score;
            const float size = fabsf(part * a1) + (p.group_top == 2 && a2 > -CUDART_INF_F ? fabsf(part * a2) : 0.f);
            const float off = a1 > -CUDART_INF_F ? 0.5f * unit + 0x1p-22f * size : 0.f;
            const float in = -redux_max(keep ? off - mine : -CUDART_INF_F);   // the lowest kept group at its lowest
            const float out = redux_max(keep ? -CUDART_INF_F : mine + off);   // the highest of the others at its highest
            if (out > -CUDART_INF_F && !(in > out)) {
                const bool open = lane < p.groups && !(keep ? mine - off > out : in > mine + off);
                const uint32_t compete = __ballot_sync(0xFFFFFFFFu, open);
                const double sum64 = softmax && !by_logit ? route_sum_f64(p, row, mx) : 1.0;
                double exact = -CUDART_INF;
                for (uint32_t left = compete; left; left &= left - 1) {
                    const int g = __ffs(left) - 1;
                    const double v = route_group_f64(p, row, g, mx, sum64);
                    if (lane == g) exact = v;
                }
                int before = __popc(kept & ~compete);
                for (uint32_t left = compete; left; left &= left - 1) {
                    const int h = __ffs(left) - 1;
                    const double v = __shfl_sync(0xFFFFFFFFu, exact, h);
                    before += (v > exact || (v == exact && h < lane)) ? 1 : 0;
                }
                kept = __ballot_sync(0xFFFFFFFFu, open ? before < p.topk_groups : keep);
            }
        }
        if (p.rows_per_group == 1) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (!((kept >> i) & 1u)) c[i] = -CUDART_INF_F;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * 32 + lane;
                if (e < E && !((kept >> (e / p.group_size)) & 1u)) c[i] = -CUDART_INF_F;
            }
        }
    }
    if (EPL > 1) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const uint32_t u = __float_as_uint(c[i] + 0.f);   // + 0: -0 and 0 are the same
            const uint32_t low = (~static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) & (EPL - 1)) ^ i;
            if (c[i] > -CUDART_INF_F) c[i] = __uint_as_float((u & ~static_cast<uint32_t>(EPL - 1)) | low);
        }
        sort_falling<EPL>(c);
    }
    float v = -CUDART_INF_F;   // lane j: the j-th largest
    uint32_t from = 0;         // and the lanes that had it; the lowest one's is taken
    const uint32_t below = (1u << lane) - 1u;
    // lane `at` takes the largest value that is left, and its lane's values move up
    const auto take = [&](int at) {
        const float m = redux_max(c[0]);
        const bool mine = c[0] == m;
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, mine);
        if (lane == at) {
            v = m;
            from = have;
        }
        if (mine && (have & below) == 0) {
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) c[i] = c[i + 1];
            c[EPL - 1] = -CUDART_INF_F;
        }
    };
    for (int j = 0; j <= k; ++j) take(j);   // lane k: the best that is left out
    const auto expert = [&] {
        const uint32_t u = __float_as_uint(v);
        return v > -CUDART_INF_F
                   ? static_cast<int>((~static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) ^ u) & (EPL - 1)) * 32 +
                         __ffs(from) - 1
                   : -1;
    };
    int id = expert(), place = lane;
    float xs = id >= 0 ? fminf(static_cast<float>(row[id]), CUDART_MAX_NORMAL_F) : 0.f;
    if (!(sizeof(LT) == 2 && by_logit)) {   // bf16 logits have the 5 bits to spare: their order is exact
        const float bs = id >= 0 && !by_logit ? p.bias[id] : 0.f;
        const float v1 = __shfl_down_sync(0xFFFFFFFFu, v, 1), x1 = __shfl_down_sync(0xFFFFFFFFu, xs, 1);
        const float b1 = __shfl_down_sync(0xFFFFFFFFu, bs, 1);
        const float tol = (by_logit ? 0x1p-120f : tol_score) + EPL * 0x1p-22f * fabsf(v);
        const bool near = lane < k && v1 > -CUDART_INF_F && v - v1 <= tol;
        bool again = near && !(by_logit ? xs >= x1 : xs == x1 && bs == b1);
        // near the border: what comes behind the best one left out must be far, too
        if (__ballot_sync(0xFFFFFFFFu, near) >> (k - 1) & 1u) {
            const float v2 = redux_max(c[0]);
            again |= lane == k - 1 && v2 > -CUDART_INF_F && v - v2 <= tol;
        }
        if (__any_sync(0xFFFFFFFFu, again)) {
            // all values that may belong to the k largest, then their order by the 64-bit values
            // (next to the lowest value, v - tol would be -inf, which every empty place reaches)
            const float last = fmaxf(__shfl_sync(0xFFFFFFFFu, v - tol, k - 1), -CUDART_MAX_NORMAL_F);
            int n = k + 1;
            for (; n < 32 && redux_max(c[0]) >= last; ++n) take(n);
            if (redux_max(c[0]) >= last) return true;   // still more of them
            id = expert();
            xs = id >= 0 ? fminf(static_cast<float>(row[id]), CUDART_MAX_NORMAL_F) : 0.f;
            const double sum64 = softmax && !by_logit ? route_sum_f64(p, row, mx) : 1.0;
            const uint64_t key = id >= 0 ? route_key_f64(p, row, id, mx, sum64) : 0;
            place = 0;
            for (int j = 0; j < n; ++j) {
                const uint64_t kj = __shfl_sync(0xFFFFFFFFu, key, j);
                const int idj = __shfl_sync(0xFFFFFFFFu, id, j);
                place += (kj > key || (kj == key && idj < id)) ? 1 : 0;
            }
            if (id < 0) place = lane < n ? lane : 32;   // behind all the others already
        }
    }
    const bool out = place < k;
    if (!out) id = -1;
    const float w = route_weight(p, p.scale, id >= 0, xs, mx, sum);
    if (out) {
        p.ids[static_cast<size_t>(t) * k + place] = id;
        p.weights[static_cast<size_t>(t) * k + place] = w;
    }
    return false;
}

// Tokens in batches of up to 32 per warp, then the batch's tokens that are done again: the 64-bit
// form is a call, and nothing of the fp32 form has to live across it.
template <typename LT, int EPL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, EPL <= 8 ? ROUTE_BLOCKS : 1) route_kernel(const __grid_constant__ RouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, step = gridDim.x * ROUTE_WARPS;
    for (long long t0 = blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5); t0 < p.T; t0 += 32LL * step) {
        uint32_t redo = 0;
        {
            float b[EPL];
            if (p.bias) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = i * 32 + lane;
                    b[i] = e < p.E ? p.bias[e] : -CUDART_INF_F;
                    if (b[i] != b[i]) report_error(p.err, ERR_DATA);
                    // +inf: the largest finite value, which has bits to spare for the index
                    b[i] = b[i] == b[i] ? fminf(b[i], CUDART_MAX_NORMAL_F) : -CUDART_INF_F;
                }
            }
            for (int n = 0; n < 32; ++n) {
                const long long t = t0 + static_cast<long long>(n) * step;
                if (t >= p.T) break;
                if (p.k > 30 || route_token<LT, EPL>(p, b, static_cast<int>(t), lane)) redo |= 1u << n;
            }
        }
        while (redo) {
            const int n = __ffs(redo) - 1;
            redo &= redo - 1;
            route_token_f64<LT>(p, static_cast<int>(t0 + static_cast<long long>(n) * step));
        }
    }
}

// Gradient of the logits from the gradient g of the weights; a warp per token, lane j the
// choice j (id -1: none). With o_j = s_j / (the chosen scores' sum):
//   softmax, renorm:  dx_j = scale·o_j·(g_j - sum_i g_i·o_i), the other logits cancel out;
//   sigmoid, renorm:  the same times (1 - s_j);
//   sigmoid:          dx_j = scale·g_j·s_j·(1 - s_j);
//   softmax:          dx_e = s_e·(scale·g_e - sum_i scale·g_i·s_i) for every e (g_e = 0 unless chosen).
// A choice that stands twice in a row adds both gradients.
// The row is first written without the choices (zeros in 16-byte stores, or the softmax term), then each choice's
// lane writes its own element: only the k chosen logits are read, except for softmax without renorm.
template <typename LT>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_backward_kernel(const __grid_constant__ RouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, E = p.E;
    const long long t = static_cast<long long>(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const LT *row = static_cast<const LT *>(p.logits) + static_cast<size_t>(t) * E;
    LT *out = static_cast<LT *>(p.grad_logits) + static_cast<size_t>(t) * E;
    int id = -1;
    float g = 0.f, x = 0.f;
    if (lane < p.k) {
        id = p.ids[static_cast<size_t>(t) * p.k + lane];
        g = p.grad_w[static_cast<size_t>(t) * p.k + lane];
        if (id >= E) {
            report_error(p.err, ERR_DATA);
            id = -1;
        }
        if (id >= 0) x = fminf(static_cast<float>(row[id]), CUDART_MAX_NORMAL_F);
    }
    const bool in = id >= 0, full = p.score == SCORE_SOFTMAX && !p.renorm;
    float mx = -CUDART_INF_F, sum = 0.f;
    if (full) {
        for (int e = lane; e < E; e += 32) mx = fmaxf(mx, route_logit(static_cast<float>(row[e]), nullptr));
        mx = redux_max(mx);
        for (int e = lane; e < E; e += 32) {
            const float v = route_logit(static_cast<float>(row[e]), nullptr);
            if (v > -CUDART_INF_F) sum += expf(v - mx);
        }
        sum = warp_sum(sum);
    }
    const float o = route_weight(p, 1.f, in, x, mx, sum);   // o_j or s_j
    const float total = warp_sum(in ? g * o : 0.f);
    float dx = in ? p.scale * (o * (p.renorm ? g - total : g)) : 0.f;
    if (in && p.score == SCORE_SIGMOID) dx *= sigmoid_scaled(-x, 0.f);
    if (full) {
        const float c = p.scale * total / sum;
        for (int e = lane; e < E; e += 32) {
            const float v = route_logit(static_cast<float>(row[e]), nullptr);
            const float d = v > -CUDART_INF_F ? -c * expf(v - mx) : 0.f;
            store_vec<LT, 1>(out + e, &d);
        }
    } else if (E * sizeof(LT) % 16 == 0) {
        for (int e = lane; e < E * static_cast<int>(sizeof(LT)) / 16; e += 32)
            reinterpret_cast<uint4 *>(out)[e] = make_uint4(0, 0, 0, 0);
    } else {
        const float zero = 0.f;
        for (int e = lane; e < E; e += 32) store_vec<LT, 1>(out + e, &zero);
    }
    // the first lane of equal ids writes their sum
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    const bool first = in && __ffs(same) - 1 == lane;
    if (__any_sync(0xFFFFFFFFu, in && !first)) {
        float s = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const float d = __shfl_sync(0xFFFFFFFFu, dx, j);
            if ((same >> j) & 1u) s += d;
        }
        dx = s;
    }
    if (full) dx -= p.scale * (total * o);
    __syncwarp();
    if (first) store_vec<LT, 1>(out + id, &dx);
}

}  // namespace dg
