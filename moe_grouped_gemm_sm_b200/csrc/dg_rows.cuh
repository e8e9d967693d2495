// dg_rows.cuh — the rows of the grouped layouts: from expert ids to rows, tokens cast into their
// k rows, and the weighted sum of the k result rows with its gradient (sm_100a).
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_norm.cuh"
#include "dg_ptx.cuh"

namespace dg {

// -----------------------------------------------------------------------------------------------
// Expert ids -> rows: a counting sort by expert, stable in the pair index t·k + j, so that the
// rows never depend on the order in which threads run.
// -----------------------------------------------------------------------------------------------
constexpr int LAYOUT_THREADS = 256, LAYOUT_WARPS = LAYOUT_THREADS / 32;
constexpr int LAYOUT_CHUNK = 2048;      // pairs a block places at least
constexpr int LAYOUT_MAX_CHUNKS = 128;
constexpr int LAYOUT_MAX_G = 1024;

struct LayoutParams {
    const int32_t *ids;        // [n]
    int32_t *dst_rows;         // [n]
    int32_t *grouped_layout;   // [M] contiguous only
    int32_t *counts;           // [G]: padded rows (contiguous), valid rows (masked)
    int32_t *hist;             // [chunks][G]
    int *err;
    int n, G, M, chunk, chunks;   // M = M_sum (contiguous) or M_max (masked)
};

// Pairs of each expert in one chunk; integer sums, so their order does not matter.
__global__ void __launch_bounds__(LAYOUT_THREADS) layout_count_kernel(const LayoutParams p) {
    extern __shared__ int s_layout[];
    pdl_launch_dependents();
    pdl_wait();
    for (int g = threadIdx.x; g < p.G; g += LAYOUT_THREADS) s_layout[g] = 0;
    __syncthreads();
    const long long i0 = static_cast<long long>(blockIdx.x) * p.chunk;
    const int end = static_cast<int>(min(static_cast<long long>(p.n), i0 + p.chunk));
    for (int i = static_cast<int>(i0) + threadIdx.x; i < end; i += LAYOUT_THREADS) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.G) atomicAdd(&s_layout[e], 1);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < p.G; g += LAYOUT_THREADS)
        p.hist[static_cast<size_t>(blockIdx.x) * p.G + g] = s_layout[g];
}

// Places one chunk's pairs. Shared memory: s_first[G] (first row of the expert), s_total[G] (its
// pairs), s_next[warps][G] (the next row of the expert for each warp's part of the chunk; a
// warp owns consecutive pairs and takes them 32 at a time, equal ids ranked by lane).
// One chunk alone counts its pairs itself, without the kernel above.
template <bool MASKED>
__global__ void __launch_bounds__(LAYOUT_THREADS) layout_place_kernel(const LayoutParams p) {
    extern __shared__ int s_layout[];
    int *s_first = s_layout, *s_total = s_layout + p.G, *s_next = s_layout + 2 * p.G;
    __shared__ int s_scan[LAYOUT_WARPS];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
    const long long i0 = static_cast<long long>(blockIdx.x) * p.chunk;
    const int end = static_cast<int>(min(static_cast<long long>(p.n), i0 + p.chunk));
    const int per = (p.chunk + LAYOUT_WARPS * 32 - 1) / (LAYOUT_WARPS * 32) * 32;   // pairs of a warp
    const int w0 = static_cast<int>(min(static_cast<long long>(end), i0 + static_cast<long long>(warp) * per));
    const int w1 = min(end, w0 + per);

    for (int g = tid; g < LAYOUT_WARPS * G; g += LAYOUT_THREADS) s_next[g] = 0;
    __syncthreads();
    for (int i = w0 + lane; i < w1; i += 32) {
        const int e = p.ids[i];
        if (e >= 0 && e < G) atomicAdd(&s_next[warp * G + e], 1);
    }
    __syncthreads();
    // totals, and the pairs of earlier chunks (kept in s_first for now)
    for (int g = tid; g < G; g += LAYOUT_THREADS) {
        int before = 0, total = 0;
        if (p.chunks == 1) {
            for (int w = 0; w < LAYOUT_WARPS; ++w) total += s_next[w * G + g];
        } else {
            for (int c = 0; c < p.chunks; ++c) {
                const int v = p.hist[static_cast<size_t>(c) * G + g];
                total += v;
                if (c < static_cast<int>(blockIdx.x)) before += v;
            }
        }
        s_total[g] = total;
        s_first[g] = before;
    }
    __syncthreads();
    // first row of each expert: masked g·M, contiguous the sum of the earlier experts' padded
    // pairs (64-bit sums are not needed: n + 127·G < 2^31)
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += LAYOUT_THREADS) {
        const int g = g0 + tid;
        int first;
        if constexpr (MASKED) {
            first = g * p.M;
        } else {
            const int padded = g < G ? (s_total[g] + 127) / 128 * 128 : 0;
            int v = padded;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) s_scan[warp] = v;
            __syncthreads();
            int base = carry;
            for (int w = 0; w < LAYOUT_WARPS; ++w) {
                if (w < warp) base += s_scan[w];
                carry += s_scan[w];
            }
            first = base + v - padded;
            __syncthreads();
            if (g < G && blockIdx.x == 0 && p.counts) p.counts[g] = max(0, min(padded, p.M - first));
        }
        if (g < G) {
            if (MASKED && blockIdx.x == 0 && p.counts) p.counts[g] = min(s_total[g], p.M);
            int next = first + s_first[g];
            s_first[g] = first;
            for (int w = 0; w < LAYOUT_WARPS; ++w) {
                const int cnt = s_next[w * G + g];
                s_next[w * G + g] = next;
                next += cnt;
            }
        }
    }
    __syncthreads();
    bool lost = false;
    for (int i = w0; i < w1; i += 32) {
        const int e0 = i + lane < w1 ? p.ids[i + lane] : -1;
        const int e = e0 >= 0 && e0 < G ? e0 : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        int row = -1;
        if (e >= 0) {
            row = s_next[warp * G + e] + __popc(same & ((1u << lane) - 1u));
            if (row >= (MASKED ? s_first[e] + p.M : p.M)) {
                row = -1;
                lost = true;
            }
        }
        __syncwarp();
        if (e >= 0 && (same >> lane) == 1u) s_next[warp * G + e] += __popc(same);   // the last of its lanes
        __syncwarp();
        if (i + lane < w1) p.dst_rows[i + lane] = row;
    }
    if (lost) report_error(p.err, ERR_DATA);
    if constexpr (!MASKED) {
        // each aligned 128-row block belongs to the last expert that starts at or before it
        if (p.grouped_layout)
            for (int b = blockIdx.x * LAYOUT_WARPS + warp; b < p.M / 128; b += gridDim.x * LAYOUT_WARPS) {
                const int r0 = b * 128;
                int lo = 0, hi = G;   // the first expert that starts behind r0 is in (lo, hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (s_first[mid] <= r0) lo = mid;
                    else hi = mid;
                }
                const int valid = s_first[lo] + s_total[lo] - r0;   // valid rows of the block
                const int r = lane * 4;
                int4 v;
                v.x = r < valid ? lo : -1;
                v.y = r + 1 < valid ? lo : -1;
                v.z = r + 2 < valid ? lo : -1;
                v.w = r + 3 < valid ? lo : -1;
                *reinterpret_cast<int4 *>(p.grouped_layout + r0 + r) = v;
            }
    }
}

// -----------------------------------------------------------------------------------------------
// The per-token FP8 cast of x [T,K] written to each token's k rows of a grouped layout of G
// groups of M rows (contiguous: G = 1, M = M_sum): row r goes to q[r] and to
// sfa[(r/M·Kb + kb)·pad4(M) + r%M]. A half-warp takes one 1x128 slice of one token.
// -----------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) cast_scatter_topk_kernel(const __nv_bfloat16 *x, const int32_t *dst, uint8_t *q,
                                                                float *sfa, int T, int k, int K, int M, int ld,
                                                                long long rows, int *err) {
    pdl_launch_dependents();
    pdl_wait();
    const int Kb = K >> 7, hl = threadIdx.x & 15;
    const long long sl = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const bool in = sl < static_cast<long long>(T) * Kb;
    const int t = in ? static_cast<int>(sl / Kb) : 0, kb = in ? static_cast<int>(sl % Kb) : 0;
    float f[8];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = ldg_stream_v4(x + static_cast<size_t>(t) * K + kb * 128 + hl * 8);
    bf16x8_to_f32(v, f);
    float m = amax8(f);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (!in) return;
    const float s = scale_of(m);
    const uint2 code = quant8(f, s);
    for (int j = 0; j < k; ++j) {
        const int r = dst[static_cast<size_t>(t) * k + j];
        if (r < 0) continue;
        if (r >= rows) {
            if (hl == 0 && kb == 0) report_error(err, ERR_DATA);
            continue;
        }
        *reinterpret_cast<uint2 *>(q + static_cast<size_t>(r) * K + kb * 128 + hl * 8) = code;
        if (hl == 0) sfa[(static_cast<size_t>(r / M) * Kb + kb) * ld + r % M] = s;
    }
}

// -----------------------------------------------------------------------------------------------
// y[t] = c[t] + sum_j w[t,j]·d[dst[t,j]] and its gradients. Rows of -1 are left out.
// -----------------------------------------------------------------------------------------------
constexpr int COMBINE_THREADS = 256, COMBINE_MAX_K = 32;

struct CombineParams {
    const __nv_bfloat16 *d;       // [R,N]
    const int32_t *dst;           // [T,k]
    const float *w;               // [T,k] or NULL (ones)
    const __nv_bfloat16 *c;       // [T,N] or NULL; may be y
    __nv_bfloat16 *y;             // [T,N]
    const __nv_bfloat16 *gy;      // backward: [T,N]
    const int32_t *layout;        // backward: [R] or NULL
    __nv_bfloat16 *gd;            // backward: [R,N] or NULL
    float *gw;                    // backward: [T,k] or NULL
    int *err;
    int T, k, N, R;
};

// The token's rows and weights in shared memory; a row outside [0, R) becomes -1.
__device__ __forceinline__ void combine_rows(const CombineParams &p, int t, int *s_row, float *s_w) {
    if (threadIdx.x < p.k) {
        int r = p.dst[static_cast<size_t>(t) * p.k + threadIdx.x];
        if (r >= p.R) {
            report_error(p.err, ERR_DATA);
            r = -1;
        }
        s_row[threadIdx.x] = r < 0 ? -1 : r;
        s_w[threadIdx.x] = p.w ? p.w[static_cast<size_t>(t) * p.k + threadIdx.x] : 1.f;
    }
    __syncthreads();
}

// Grid (T, column parts): a block takes the vectors of 8 columns y·blockDim.x + threadIdx.x, ...
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(const CombineParams p) {
    __shared__ int s_row[COMBINE_MAX_K];
    __shared__ float s_w[COMBINE_MAX_K];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x;
    combine_rows(p, t, s_row, s_w);
    for (int i = blockIdx.y * COMBINE_THREADS + threadIdx.x; i < p.N / 8; i += gridDim.y * COMBINE_THREADS) {
        float acc[8];
        if (p.c) {
            load_vec<__nv_bfloat16, 8>(p.c + static_cast<size_t>(t) * p.N + static_cast<size_t>(i) * 8, acc);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        }
        for (int j = 0; j < p.k; ++j) {
            if (s_row[j] < 0) continue;
            float f[8];
            bf16x8_to_f32(ldg_stream_v4(p.d + static_cast<size_t>(s_row[j]) * p.N + static_cast<size_t>(i) * 8), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(s_w[j], f[e], acc[e]);
        }
        store_vec<__nv_bfloat16, 8>(p.y + static_cast<size_t>(t) * p.N + static_cast<size_t>(i) * 8, acc);
    }
}

// Blocks 0 .. T-1: gd[dst[t,j]] = w[t,j]·gy[t] and gw[t,j] = <gy[t], d[dst[t,j]]> (0 for a row of
// -1). The blocks behind them (with a layout) zero the rows of gd whose layout entry is negative.
__global__ void __launch_bounds__(COMBINE_THREADS) combine_backward_kernel(const CombineParams p) {
    __shared__ int s_row[COMBINE_MAX_K];
    __shared__ float s_w[COMBINE_MAX_K];
    __shared__ float s_red[32];
    pdl_launch_dependents();
    pdl_wait();
    const int nv = p.N / 8;
    if (blockIdx.x >= p.T) {
        for (int r = blockIdx.x - p.T; r < p.R; r += gridDim.x - p.T) {
            if (p.layout[r] >= 0) continue;
            uint4 *row = reinterpret_cast<uint4 *>(p.gd + static_cast<size_t>(r) * p.N);
            for (int i = threadIdx.x; i < nv; i += COMBINE_THREADS) row[i] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const int t = blockIdx.x;
    combine_rows(p, t, s_row, s_w);
    const __nv_bfloat16 *gy = p.gy + static_cast<size_t>(t) * p.N;
    for (int j = 0; j < p.k; ++j) {
        const int r = s_row[j];
        float dot = 0.f;
        if (r >= 0)
            for (int i = threadIdx.x; i < nv; i += COMBINE_THREADS) {
                float g[8], f[8];
                load_vec<__nv_bfloat16, 8>(gy + static_cast<size_t>(i) * 8, g);
                if (p.gw) {
                    bf16x8_to_f32(ldg_stream_v4(p.d + static_cast<size_t>(r) * p.N + static_cast<size_t>(i) * 8), f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot = fmaf(g[e], f[e], dot);
                }
                if (p.gd) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] *= s_w[j];
                    store_vec<__nv_bfloat16, 8>(p.gd + static_cast<size_t>(r) * p.N + static_cast<size_t>(i) * 8, g);
                }
            }
        if (p.gw) {
            const float s = row_sum(dot, s_red);
            if (threadIdx.x == 0) p.gw[static_cast<size_t>(t) * p.k + j] = s;
            __syncthreads();
        }
    }
}

}  // namespace dg
