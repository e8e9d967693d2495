// dg_norm.cuh — layer norm and RMS norm: forward (with an optional per-token FP8 cast of the
// result), and backward with the reduction of the weight's and the bias's gradients (sm_100a).
//
// Forward, row by row over K elements:
//   mu = mean(x) (0 in the RMS form), r = 1/sqrt(mean((x - mu)^2) + eps), xh = (x - mu)·r,
//   y = xh·w + b.
// Backward, with u = dy·w:
//   dx = r·(u - mean(u) - xh·mean(u·xh))   (RMS: without mean(u)),
//   dw = sum over rows of dy·xh,   db = sum over rows of dy.
// Sums, statistics and the gradients of w and b are fp32; a result is rounded once, to x's type.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_cast.cuh"
#include "dg_ptx.cuh"

namespace dg {

// V consecutive elements as fp32. V = 1 takes any element; larger V needs the address aligned to
// the vector's size.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float *f) {
    if constexpr (V == 1) {
        f[0] = static_cast<float>(*p);
    } else if constexpr (sizeof(T) == 2) {
        static_assert(V == 4 || V == 8, "bf16 vector");
        if constexpr (V == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            f[0] = __uint_as_float(v.x << 16);
            f[1] = __uint_as_float(v.x & 0xFFFF0000u);
            f[2] = __uint_as_float(v.y << 16);
            f[3] = __uint_as_float(v.y & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p)[i];
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float *f) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(f[0]);
        else *p = f[0];
    } else if constexpr (sizeof(T) == 2) {
        static_assert(V == 8, "bf16 vector");
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the blockDim.x threads of a row, the same bits in every thread. One warp a row needs no
// barrier; otherwise the row is the whole block and `red` (32 floats) must not be in use.
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if (blockDim.x == 32) return v;
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += red[i];
    return s;
}

constexpr int NORM_MAX_THREADS = 1024, NORM_DX_MAX_THREADS = 512;   // threads of a row

struct NormParams {
    const void *x, *w, *b;   // w, b may be NULL (ones, zeros)
    void *y;                 // may be NULL
    uint8_t *q;              // e4m3 codes, may be NULL
    float *sfa;              // with q: [K/128][ld]
    float *mean, *rstd;      // [T], may be NULL
    int T, K, ld, rms;
    float eps;
};

// One row of K elements per blockDim.x threads (blockDim.y rows per block, one warp each when
// blockDim.y > 1). Thread t holds the vectors t, t + blockDim.x, ... of V elements in registers: x is
// read once, the mean and then the mean square of the differences are taken from registers.
// With q: the 128 / V threads that hold one 128-element slice take its amax by shuffles; the
// codes are those of the unrounded fp32 y (one rounding instead of two).
template <typename XT, typename WT, int V, int VPT>
__global__ void __launch_bounds__(NORM_MAX_THREADS) layer_norm_kernel(const NormParams p) {
    __shared__ float s_red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.T) return;   // blockDim.y > 1 only with one warp a row: no barrier follows
    const int K = p.K, nv = K / V, nt = blockDim.x;
    const XT *x = static_cast<const XT *>(p.x) + static_cast<size_t>(row) * K;
    float f[VPT][V];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = j * nt + threadIdx.x;
        if (i < nv) {
            load_vec<XT, V>(x + static_cast<size_t>(i) * V, f[j]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) f[j][e] = 0.f;
        }
    }
    float mu = 0.f;
    if (!p.rms) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) s += f[j][e];
        mu = row_sum(s, s_red[0]) / static_cast<float>(K);
    }
    float s2 = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (j * nt + threadIdx.x < nv) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f[j][e] -= mu;
                s2 += f[j][e] * f[j][e];
            }
        }
    const float r = 1.f / sqrtf(row_sum(s2, s_red[1]) / static_cast<float>(K) + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = r;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = j * nt + threadIdx.x;
        if (i < nv) {
            float w[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[j][e] *= r;
            if (p.w) {
                load_vec<WT, V>(static_cast<const WT *>(p.w) + static_cast<size_t>(i) * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) f[j][e] *= w[e];
            }
            if (p.b) {
                load_vec<WT, V>(static_cast<const WT *>(p.b) + static_cast<size_t>(i) * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) f[j][e] += w[e];
            }
            if (p.y) store_vec<XT, V>(static_cast<XT *>(p.y) + static_cast<size_t>(row) * K + static_cast<size_t>(i) * V, f[j]);
        }
        if constexpr (V > 1) {
            if (p.q) {   // K % 128 == 0: the threads of a slice are all inside the row or all outside
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) m = fmaxf(m, fabsf(f[j][e]));
#pragma unroll
                for (int o = 64 / V; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                if (i < nv) {
                    const float sc = scale_of(m);
                    uint8_t *q = p.q + static_cast<size_t>(row) * K + static_cast<size_t>(i) * V;
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2 *>(q) = quant8(f[j], sc);
                    else
                        *reinterpret_cast<uint32_t *>(q) = quant4(f[j], sc);
                    const int per = 128 / V;
                    if (i % per == 0) p.sfa[static_cast<size_t>(i / per) * p.ld + row] = sc;
                }
            }
        }
    }
}

struct NormBackParams {
    const void *dy, *x, *w;
    const float *mean, *rstd;   // mean NULL = the RMS form
    void *dx;
    float *part;                // [parts][2 or 1][K] column sums (dw, then db)
    float *dw, *db;             // may be NULL
    int T, K, parts;
};

// dx of one row per blockDim.x threads, laid out as in the forward kernel.
template <typename XT, typename WT, int V, int VPT>
__global__ void __launch_bounds__(NORM_DX_MAX_THREADS) layer_norm_dx_kernel(const NormBackParams p) {
    __shared__ float s_red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.T) return;
    const int K = p.K, nv = K / V, nt = blockDim.x;
    const size_t at = static_cast<size_t>(row) * K;
    const float mu = p.mean ? p.mean[row] : 0.f, r = p.rstd[row];
    float u[VPT][V], xh[VPT][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = j * nt + threadIdx.x;
        if (i < nv) {
            load_vec<XT, V>(static_cast<const XT *>(p.x) + at + static_cast<size_t>(i) * V, xh[j]);
            load_vec<XT, V>(static_cast<const XT *>(p.dy) + at + static_cast<size_t>(i) * V, u[j]);
            float w[V];
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = 1.f;
            if (p.w) load_vec<WT, V>(static_cast<const WT *>(p.w) + static_cast<size_t>(i) * V, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                xh[j][e] = (xh[j][e] - mu) * r;
                u[j][e] *= w[e];
                s1 += u[j][e];
                s2 += u[j][e] * xh[j][e];
            }
        }
    }
    const float c1 = p.mean ? row_sum(s1, s_red[0]) / static_cast<float>(K) : 0.f;
    const float c2 = row_sum(s2, s_red[1]) / static_cast<float>(K);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = j * nt + threadIdx.x;
        if (i < nv) {
#pragma unroll
            for (int e = 0; e < V; ++e) u[j][e] = r * (u[j][e] - c1 - xh[j][e] * c2);
            store_vec<XT, V>(static_cast<XT *>(p.dx) + at + static_cast<size_t>(i) * V, u[j]);
        }
    }
}

// Column sums over one part of the rows: block (32, 8), a thread a column, 8 rows at a time;
// grid (ceil(K/32), parts).
template <typename XT>
__global__ void __launch_bounds__(256) layer_norm_dwdb_kernel(const NormBackParams p) {
    __shared__ float s_w[8][32], s_b[8][32];
    pdl_launch_dependents();
    pdl_wait();
    const int col = blockIdx.x * 32 + threadIdx.x;
    float aw = 0.f, ab = 0.f;
    if (col < p.K)
        for (int t = blockIdx.y * 8 + threadIdx.y; t < p.T; t += 8 * p.parts) {
            const size_t at = static_cast<size_t>(t) * p.K + col;
            const float dy = static_cast<float>(static_cast<const XT *>(p.dy)[at]);
            const float xv = static_cast<float>(static_cast<const XT *>(p.x)[at]);
            aw += dy * ((xv - (p.mean ? p.mean[t] : 0.f)) * p.rstd[t]);
            ab += dy;
        }
    s_w[threadIdx.y][threadIdx.x] = aw;
    s_b[threadIdx.y][threadIdx.x] = ab;
    __syncthreads();
    if (threadIdx.y == 0 && col < p.K) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            aw += s_w[i][threadIdx.x];
            ab += s_b[i][threadIdx.x];
        }
        p.part[(static_cast<size_t>(blockIdx.y) * 2) * p.K + col] = aw;
        p.part[(static_cast<size_t>(blockIdx.y) * 2 + 1) * p.K + col] = ab;
    }
}

// dw and db from the parts, added in the parts' order: a thread a column.
__global__ void __launch_bounds__(256) layer_norm_parts_kernel(const NormBackParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= p.K) return;
    float aw = 0.f, ab = 0.f;
    for (int i = 0; i < p.parts; ++i) {
        aw += p.part[(static_cast<size_t>(i) * 2) * p.K + col];
        ab += p.part[(static_cast<size_t>(i) * 2 + 1) * p.K + col];
    }
    if (p.dw) p.dw[col] = aw;
    if (p.db) p.db[col] = ab;
}

}  // namespace dg
