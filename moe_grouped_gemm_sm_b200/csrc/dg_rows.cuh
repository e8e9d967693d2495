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
//
// One cluster of up to 16 blocks does it in one launch and without scratch in global memory: each block
// counts its consecutive pairs per warp and expert, the blocks read each other's counts through distributed
// shared memory, and each places its own pairs. Latency-bound throughout (131072 pairs over 256 experts are
// 0.3 us of traffic, and take 10.8 us; 1024 pairs 3.0); two launches over 64 blocks with the counts in global
// memory took 14 to 17 us, and needed scratch.
// Equal ids of a warp are found by one ballot per bit of the id (BITS, unrolled); the match instruction took some
// 400 cycles.
// -----------------------------------------------------------------------------------------------
constexpr int LAYOUT_MAX_WARPS = 32, LAYOUT_MAX_CLUSTER = 16, LAYOUT_MAX_G = 1024;

struct LayoutParams {
    const int32_t *ids;        // [n]
    int32_t *dst_rows;         // [n]
    int32_t *grouped_layout;   // [M] contiguous only
    int32_t *counts;           // [G]: padded rows (contiguous), valid rows (masked)
    int *err;
    int n, G, M;               // M = M_sum (contiguous) or M_max (masked)
    int per_warp;              // consecutive pairs of a warp, a multiple of 32
};

__device__ __forceinline__ int ld_shared_cluster(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Shared memory: s_first[G] (first row of the expert), s_total[G] (its pairs), s_count[G] (those of this block, read
// by the others), s_next[warps][G] (a warp's pairs, then its next row of the expert; masked its next place among the
// expert's rows, since g·M plus the pairs of an expert that has too many may pass 2^31).
template <bool MASKED, int BITS>
__global__ void __launch_bounds__(32 * LAYOUT_MAX_WARPS) layout_kernel(const __grid_constant__ LayoutParams p) {
    extern __shared__ int s_layout[];
    const int G = p.G;
    int *s_first = s_layout, *s_total = s_first + G, *s_count = s_total + G, *s_next = s_count + G;
    __shared__ int s_scan[LAYOUT_MAX_WARPS];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
    const int blocks = gridDim.x, rank = blockIdx.x;   // the grid is one cluster
    const long long start = (static_cast<long long>(rank) * warps + warp) * p.per_warp;
    const int w0 = static_cast<int>(min(static_cast<long long>(p.n), start));
    const int w1 = static_cast<int>(min(static_cast<long long>(p.n), start + p.per_warp));

    for (int g = tid; g < warps * G; g += nt) s_next[g] = 0;
    __syncthreads();
    for (int i = w0 + lane; i < w1; i += 128) {   // four loads under way at a time
        int e[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) e[q] = i + 32 * q < w1 ? p.ids[i + 32 * q] : -1;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (e[q] >= 0 && e[q] < G) atomicAdd(&s_next[warp * G + e[q]], 1);
    }
    __syncthreads();
    for (int g = tid; g < G; g += nt) {
        int count = 0;
        for (int w = 0; w < warps; ++w) count += s_next[w * G + g];
        s_count[g] = count;
    }
    if (blocks > 1) cluster_sync();
    // first row of each expert: masked g·M, contiguous the sum of the earlier experts' padded
    // pairs (64-bit sums are not needed: n + 127·G < 2^31)
    int carry = 0;
    for (int g0 = 0; g0 < G; g0 += nt) {
        const int g = g0 + tid;
        int total = 0, before = 0;   // pairs of the expert, and those in earlier blocks
        if (g < G) {
            if (blocks > 1) {
                const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(s_count + g));
#pragma unroll
                for (int c = 0; c < LAYOUT_MAX_CLUSTER; ++c) {
                    const int v = c < blocks ? ld_shared_cluster(mapa_shared(mine, c)) : 0;
                    total += v;
                    if (c < rank) before += v;
                }
            } else {
                total = s_count[g];
            }
            s_total[g] = total;
        }
        int first;
        if constexpr (MASKED) {
            first = g * p.M;
        } else {
            const int padded = (total + 127) / 128 * 128;
            int v = padded;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) s_scan[warp] = v;
            __syncthreads();
            const int sum = lane < warps ? s_scan[lane] : 0;
            first = carry + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0) + v - padded;
            carry += __reduce_add_sync(0xFFFFFFFFu, sum);
            __syncthreads();
            if (g < G && rank == 0 && p.counts) p.counts[g] = max(0, min(padded, p.M - first));
        }
        if (g < G) {
            if (MASKED && rank == 0 && p.counts) p.counts[g] = min(total, p.M);
            s_first[g] = first;
            int next = MASKED ? before : first + before;
            for (int w = 0; w < warps; ++w) {
                const int count = s_next[w * G + g];
                s_next[w * G + g] = next;
                next += count;
            }
        }
    }
    // this block has read the others' counts; none of them may leave before all have
    if (blocks > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    __syncthreads();
    bool lost = false;
    for (int i = w0; i < w1; i += 32) {
        const int e = i + lane < w1 ? p.ids[i + lane] : -1;
        const bool in = e >= 0 && e < G;
        uint32_t same = __ballot_sync(0xFFFFFFFFu, in);
#pragma unroll
        for (int b = 0; b < BITS; ++b) {
            const int bit = (e << (31 - b)) >> 31;   // all ones or zero
            same &= ~(__ballot_sync(0xFFFFFFFFu, bit != 0) ^ static_cast<uint32_t>(bit));
        }
        int row = -1;
        if (in) {
            row = s_next[warp * G + e] + __popc(same & ((1u << lane) - 1u));
            if (row >= p.M) {
                row = -1;
                lost = true;
            } else if (MASKED) {
                row += s_first[e];
            }
        }
        __syncwarp();
        if (in && (same >> lane) == 1u) s_next[warp * G + e] += __popc(same);   // the last of its lanes
        __syncwarp();
        if (i + lane < w1) p.dst_rows[i + lane] = row;
    }
    if (lost) report_error(p.err, ERR_DATA);
    if constexpr (!MASKED) {
        // Each aligned 128-row block belongs to the last expert that starts at or before it. A warp takes every
        // all-th block, 32 at a time: each lane looks up one, then the warp writes them one after another.
        const int all = blocks * warps, n128 = p.M / 128;
        for (int b0 = rank * warps + warp; b0 < n128; b0 += 32 * all) {
            const int r0 = min(b0 + lane * all, n128 - 1) * 128;
            int lo = 0, hi = G;   // the first expert that starts behind r0 is in (lo, hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_first[mid] <= r0) lo = mid;
                else hi = mid;
            }
            const int end = s_first[lo] + s_total[lo];   // of the expert's valid rows
            for (int q = 0; q < 32 && b0 + q * all < n128; ++q) {
                const int g = __shfl_sync(0xFFFFFFFFu, lo, q), stop = __shfl_sync(0xFFFFFFFFu, end, q);
                const int r = (b0 + q * all) * 128 + lane * 4;
                int4 v;
                v.x = r < stop ? g : -1;
                v.y = r + 1 < stop ? g : -1;
                v.z = r + 2 < stop ? g : -1;
                v.w = r + 3 < stop ? g : -1;
                *reinterpret_cast<int4 *>(p.grouped_layout + r) = v;
            }
        }
    }
    if (blocks > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// -----------------------------------------------------------------------------------------------
// The per-token FP8 cast of x [T,K] written to each token's k rows of a grouped layout of G
// groups of M rows (contiguous: G = 1, M = M_sum): row r goes to q[r] and to
// sfa[(r/M·Kb + kb)·pad4(M) + r%M]. Bound by its writes: k·K bytes a token, 2·K are read.
//
// Grid (T, parts of K): a block takes one token's 16-element pieces, one a thread (8 lanes a 1x128 slice),
// quantises them once and stores 16 bytes to each row. 4 blocks of 224 threads an SM, with registers for the next
// piece's loads: 4096 tokens x 7168 to 8 rows take 58.8 us (78 % of the copy rate); blocks of 448 65.4, and with
// registers for 6 of 224 63.7 (and 7.0 instead of 4.8 for 128 tokens). The scales of a warp's 4 slices go out 8 rows at a time:
// lane l writes slice l/8's scale to the (l%8)-th row.
// -----------------------------------------------------------------------------------------------
constexpr int SCATTER_THREADS = 224, SCATTER_ROWS = 64;   // rows of a token held in shared memory at a time

__global__ void __launch_bounds__(SCATTER_THREADS, 4) cast_scatter_topk_kernel(const __nv_bfloat16 *x, const int32_t *dst,
                                                                            uint8_t *q, float *sfa, int k, int K, int M,
                                                                            int ld, long long rows, int *err) {
    __shared__ int s_row[SCATTER_ROWS];
    __shared__ long long s_sf[SCATTER_ROWS];
    pdl_launch_dependents();
    pdl_wait();
    const int Kb = K >> 7, t = blockIdx.x, lane = threadIdx.x & 31;
    for (int j0 = 0; j0 < k; j0 += SCATTER_ROWS) {
        const int n = min(k - j0, SCATTER_ROWS);
        // a warp's pieces are 4 whole slices (K % 128 == 0): lanes beyond K come 8 at a time. The first piece is
        // on its way while the rows are looked up.
        int i0 = (blockIdx.y * blockDim.x + (threadIdx.x & ~31)) * 16;
        uint4 v0, v1;
        const auto fetch = [&] {
            const int i = i0 + lane * 16;
            const __nv_bfloat16 *at = x + static_cast<size_t>(t) * K + i;
            v0 = v1 = make_uint4(0, 0, 0, 0);
            if (i < K) {
                v0 = ldg_stream_v4(at);
                v1 = ldg_stream_v4(at + 8);
            }
        };
        fetch();
        if (j0) __syncthreads();
        for (int j = threadIdx.x; j < n; j += blockDim.x) {   // a block may have fewer threads than rows
            int r = dst[static_cast<size_t>(t) * k + j0 + j];
            if (r >= rows) {
                if (blockIdx.y == 0) report_error(err, ERR_DATA);
                r = -1;
            }
            s_row[j] = r;
            s_sf[j] = r < 0 ? -1 : static_cast<long long>(r / M) * Kb * ld + r % M;
        }
        __syncthreads();
        while (i0 < K) {
            const int i = i0 + lane * 16;
            const bool in = i < K;
            float f[2][8];
            bf16x8_to_f32(v0, f[0]);
            bf16x8_to_f32(v1, f[1]);
            i0 += gridDim.y * blockDim.x * 16;
            if (i0 < K) fetch();
            float m = fmaxf(amax8(f[0]), amax8(f[1]));
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float s = scale_of(m);
            const uint2 c0 = quant8(f[0], s), c1 = quant8(f[1], s);
            const uint4 code = make_uint4(c0.x, c0.y, c1.x, c1.y);
            if (!in) continue;
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const int r = s_row[j];
                if (r >= 0) *reinterpret_cast<uint4 *>(q + static_cast<size_t>(r) * K + i) = code;
            }
            for (int j = lane & 7; j < n; j += 8) {
                const long long at = s_sf[j];
                if (at >= 0) sfa[at + static_cast<long long>(i >> 7) * ld] = s;
            }
        }
    }
}

// -----------------------------------------------------------------------------------------------
// y[t] = c[t] + sum_j w[t,j]·d[dst[t,j]] and its gradients. Rows of -1 are left out.
// -----------------------------------------------------------------------------------------------
constexpr int COMBINE_THREADS = 256, COMBINE_MAX_K = 32;
constexpr int BACK_ROWS = 4;   // rows that a block of the backward pass has under way

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

// Grid (T, column parts): a block takes the vectors of 8 columns y·blockDim.x + threadIdx.x, .... HBM-bound: the
// loads of 8 rows are under way before the first is used (one at a time, 128 tokens of 8 rows took 5.9 us, so
// 4.4). 4096 tokens x 7168 from 8 rows: 83.7 us, 97 % of the copy rate; with fewer registers (6 blocks an SM) 150.
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(const __grid_constant__ CombineParams p) {
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
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (j0 + q < p.k && s_row[j0 + q] >= 0)
                    v[q] = ldg_stream_v4(p.d + static_cast<size_t>(s_row[j0 + q]) * p.N + static_cast<size_t>(i) * 8);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (j0 + q < p.k && s_row[j0 + q] >= 0) {
                    float f[8];
                    bf16x8_to_f32(v[q], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(s_w[j0 + q], f[e], acc[e]);
                }
        }
        store_vec<__nv_bfloat16, 8>(p.y + static_cast<size_t>(t) * p.N + static_cast<size_t>(i) * 8, acc);
    }
}

// Blocks 0 .. T-1: gd[dst[t,j]] = w[t,j]·gy[t] and gw[t,j] = <gy[t], d[dst[t,j]]> (0 for a row of
// -1), BACK_ROWS rows at a time: gy is read once for them, their loads are under way together, and their dot
// products share one reduction. The blocks behind them (with a layout) zero the rows of gd whose layout entry is
// negative. HBM-bound, half reads and half writes: 4096 x 7168, 8 rows: 197 us, 87 % of the copy rate (8 rows at a
// time: 247, with too few blocks an SM).
__global__ void __launch_bounds__(COMBINE_THREADS, 6) combine_backward_kernel(const __grid_constant__ CombineParams p) {
    __shared__ int s_row[COMBINE_MAX_K];
    __shared__ float s_w[COMBINE_MAX_K];
    __shared__ float s_dot[COMBINE_THREADS / 32][BACK_ROWS];
    pdl_launch_dependents();
    pdl_wait();
    const int nv = p.N / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) >= p.T) {
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
    for (int j0 = 0; j0 < p.k; j0 += BACK_ROWS) {
        float dot[BACK_ROWS];
#pragma unroll
        for (int q = 0; q < BACK_ROWS; ++q) dot[q] = 0.f;
        for (int i = threadIdx.x; i < nv; i += COMBINE_THREADS) {
            uint4 v[BACK_ROWS];
            if (p.gw) {
#pragma unroll
                for (int q = 0; q < BACK_ROWS; ++q)
                    if (j0 + q < p.k && s_row[j0 + q] >= 0)
                        v[q] = ldg_stream_v4(p.d + static_cast<size_t>(s_row[j0 + q]) * p.N + static_cast<size_t>(i) * 8);
            }
            float g[8];
            load_vec<__nv_bfloat16, 8>(gy + static_cast<size_t>(i) * 8, g);
#pragma unroll
            for (int q = 0; q < BACK_ROWS; ++q) {
                if (j0 + q >= p.k || s_row[j0 + q] < 0) continue;
                if (p.gw) {
                    float f[8];
                    bf16x8_to_f32(v[q], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[q] = fmaf(g[e], f[e], dot[q]);
                }
                if (p.gd) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = g[e] * s_w[j0 + q];
                    store_vec<__nv_bfloat16, 8>(p.gd + static_cast<size_t>(s_row[j0 + q]) * p.N + static_cast<size_t>(i) * 8, o);
                }
            }
        }
        if (p.gw) {
            if (j0) __syncthreads();   // the last BACK_ROWS rows' sums have been read
#pragma unroll
            for (int q = 0; q < BACK_ROWS; ++q) {
                const float s = warp_sum(dot[q]);
                if (lane == q) s_dot[warp][q] = s;
            }
            __syncthreads();
            if (threadIdx.x < BACK_ROWS && j0 + static_cast<int>(threadIdx.x) < p.k) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < COMBINE_THREADS / 32; ++w) s += s_dot[w][threadIdx.x];
                p.gw[static_cast<size_t>(t) * p.k + j0 + threadIdx.x] = s;
            }
        }
    }
}

}  // namespace dg
