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

// Two fp32 values in one register pair, for the packed fp32 instructions (each half rounded as the
// scalar instruction rounds): they halve the arithmetic instructions of the row kernels.
struct Pair {
    float2 v;
};
__device__ __forceinline__ Pair pair(float lo, float hi) { return Pair{make_float2(lo, hi)}; }
__device__ __forceinline__ float2 halves(Pair p) { return p.v; }
__device__ __forceinline__ Pair operator+(Pair a, Pair b) { return Pair{__fadd2_rn(a.v, b.v)}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) { return Pair{__fmul2_rn(a.v, b.v)}; }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) { return Pair{__ffma2_rn(a.v, b.v, c.v)}; }

template <typename T, int V>
__device__ __forceinline__ void load_pairs(const T *p, Pair *f) {
    float s[V];
    load_vec<T, V>(p, s);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) f[e] = pair(s[2 * e], s[2 * e + 1]);
}
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T *p, const Pair *f) {
    float s[V];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
        const float2 h = halves(f[e]);
        s[2 * e] = h.x;
        s[2 * e + 1] = h.y;
    }
    store_vec<T, V>(p, s);
}

// The warp's sums of a and of b, in every lane: halves of the warp take one value each after the
// first exchange.
__device__ __forceinline__ float2 warp_sum2(float a, float b) {
    const bool up = (threadIdx.x & 16) != 0;
    float v = (up ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    return up ? make_float2(w, v) : make_float2(v, w);
}

// The warp's sums of the four parts of v: lane 8·i holds the i-th.
__device__ __forceinline__ float warp_sum4_spread(float4 v) {
    const bool up = (threadIdx.x & 16) != 0, up8 = (threadIdx.x & 8) != 0;
    const float a = (up ? v.z : v.x) + __shfl_xor_sync(0xFFFFFFFFu, up ? v.x : v.z, 16);
    const float b = (up ? v.w : v.y) + __shfl_xor_sync(0xFFFFFFFFu, up ? v.y : v.w, 16);
    float s = (up8 ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, up8 ? a : b, 8);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
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

// s / n from inv = 1/n. The product with the rounded reciprocal alone may miss the quotient by a unit in the last
// place, and a row of equal values would then have a deviation: 7168 times 3 gave a mean of 3.0000002. The
// remainder s - q·n is exact in one fma, and the second one adds what is missing (Markstein's correction of a
// quotient): three instructions, once a row. A sum that is not finite gives NaN: its row has no finite result anyway.
__device__ __forceinline__ float mean_of(float s, float n, float inv) {
    const float q = s * inv;
    return fmaf(fmaf(-q, n, s), inv, q);
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

// The cast epilogue of vector i of a row: the 128 / V threads that hold one 1x128 slice take its amax (m:
// the vector's) by shuffles, so all lanes of a warp call it. The codes are those of the unrounded
// fp32 values (one rounding instead of two).
template <int V>
__device__ __forceinline__ void norm_cast(const NormParams &p, const float (&f)[V], float m, long long row, int i, int nv) {
#pragma unroll
    for (int o = 64 / V; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (i >= nv) return;
    const float sc = scale_of(m);
    uint8_t *q = p.q + static_cast<size_t>(row) * p.K + static_cast<size_t>(i) * V;
    if constexpr (V == 8)
        *reinterpret_cast<uint2 *>(q) = quant8(f, sc);
    else
        *reinterpret_cast<uint32_t *>(q) = quant4(f, sc);
    constexpr int per = 128 / V;
    if (i % per == 0) p.sfa[static_cast<size_t>(i / per) * p.ld + row] = sc;
}

// One row of K elements per blockDim.x threads (blockDim.y rows per block, one warp each when
// blockDim.y > 1). Thread t holds the vectors t, t + blockDim.x, ... of V elements in registers: x is
// read once, the mean and then the mean square of the differences are taken from registers. For few rows, where the
// latency of one row counts (16 x 7168 with the cast: 2.9 us), for rows of up to 128 and for rows longer than a
// ring (below).
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
    // within 2 ulp, where a root and a quotient would be within 1; the sum of K squares weighs more
    const float r = rsqrtf(row_sum(s2, s_red[1]) / static_cast<float>(K) + p.eps);
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
            XT *y = static_cast<XT *>(p.y) + static_cast<size_t>(row) * K + static_cast<size_t>(i) * V;
            if (p.y) store_vec<XT, V>(y, f[j]);
        }
        if constexpr (V > 1) {
            if (p.q) {   // K % 128 == 0: the threads of a slice are all inside the row or all outside
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) m = fmaxf(m, fabsf(f[j][e]));
                norm_cast<V>(p, f[j], m, row, i, nv);
            }
        }
    }
}

// Rows in a ring of shared memory per team of threads, for many rows. blockDim.x threads (a team) share a
// row; every thread owns N columns of it (NormColumns), the same ones for every row that its team takes.
// blockDim.y > 1 teams of one warp each serve short rows. The ring has NORM_STAGES stages of R rows (of one or
// two tensors) and is filled two stages ahead by cp.async; R rows share their barriers.
// COLS_VECTORS: K is a whole number of 16-byte vectors; a thread owns vectors of V columns, copies and reads its own
// only, and the ring needs no barrier. COLS_EXACT: and K = N·blockDim.x, so that nothing needs a bounds check (the
// checks' zero registers and branches were a quarter of the backward pass's instructions). COLS_SINGLE: rows begin
// anywhere in the tensor (which starts on 16 bytes): a stage takes the 16-byte chunks that hold its row (the bytes
// behind the tensor's end as zeros), a thread owns single columns blockDim.x apart, and a barrier stands between the
// copies and the reads.
enum : int { COLS_SINGLE = 0, COLS_VECTORS = 1, COLS_EXACT = 2 };
constexpr int NORM_STAGES = 3, NORM_RING_THREADS = 512;   // 512 threads an SM leave 128 registers each

__device__ __forceinline__ void cp_async16(uint32_t smem, const void *gmem, int bytes = 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}

template <typename XT, int N, int COLS>
struct NormColumns {
    static constexpr bool VEC = COLS != COLS_SINGLE;
    static constexpr int C = 16 / static_cast<int>(sizeof(XT));   // elements of 16 bytes
    static constexpr int V = VEC ? C : 1;
    static constexpr int VPT = N / V;                             // vectors (single columns) of a thread
    int K, nt, tid;
    __device__ __forceinline__ explicit NormColumns(int k) : K(k), nt(blockDim.x), tid(threadIdx.x) {}

    // elements between two rows of the ring
    static __host__ __device__ __forceinline__ int pitch(int K) { return VEC ? K : (K + 2 * C - 2) / C * C; }
    // where a row that starts at element `at` of its tensor begins within its place
    __device__ __forceinline__ int offset(size_t at) const { return VEC ? 0 : static_cast<int>(at % C); }

    // one row, which starts at element `at` of a tensor of `total`, into its place of the ring
    __device__ __forceinline__ void fetch(XT *slot, const XT *x, size_t at, size_t total) const {
        const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(slot));
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = (j * nt + tid) * V;
                if (COLS == COLS_EXACT || i < K) cp_async16(s + i * static_cast<int>(sizeof(XT)), x + at + i);
            }
        } else {
            const size_t first = at / C * C;
            for (int i = tid * C; first + i < at + K; i += nt * C) {
                const size_t left = (total - first - i) * sizeof(XT);
                cp_async16(s + i * static_cast<int>(sizeof(XT)), x + first + i, left < 16 ? static_cast<int>(left) : 16);
            }
        }
    }
    // the thread's columns of a row, 0 where it has none
    template <typename T>
    __device__ __forceinline__ void load(const T *row, Pair (&f)[N / 2]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = (j * nt + tid) * V;
                if (COLS == COLS_EXACT || i < K) {
                    load_pairs<T, V>(row + i, f + j * (V / 2));
                } else {
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) f[j * (V / 2) + e] = pair(0.f, 0.f);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const int i = 2 * e * nt + tid, i2 = i + nt;
                f[e] = pair(i < K ? static_cast<float>(row[i]) : 0.f, i2 < K ? static_cast<float>(row[i2]) : 0.f);
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, const Pair (&f)[N / 2]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = (j * nt + tid) * V;
                if (COLS == COLS_EXACT || i < K) store_pairs<T, V>(row + i, f + j * (V / 2));
            }
        } else {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const int i = 2 * e * nt + tid, i2 = i + nt;
                const float2 h = halves(f[e]);
                if (i < K) store_vec<T, 1>(row + i, &h.x);
                if (i2 < K) store_vec<T, 1>(row + i2, &h.y);
            }
        }
    }
    // sum over the thread's columns of (f - mu)^2
    __device__ __forceinline__ float squares(const Pair (&f)[N / 2], float mu) const {
        const Pair c = pair(-mu, -mu);
        if constexpr (VEC) {
            Pair q = pair(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (COLS == COLS_EXACT || (j * nt + tid) * V < K) {
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        const Pair d = f[j * (V / 2) + e] + c;
                        q = fma2(d, d, q);
                    }
                }
            const float2 h = halves(q);
            return h.x + h.y;
        } else {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const int i = 2 * e * nt + tid;
                const float2 h = halves(f[e] + c);
                if (i < K) q = fmaf(h.x, h.x, q);
                if (i + nt < K) q = fmaf(h.y, h.y, q);
            }
            return q;
        }
    }
    // columns that warp `w` of the team owns
    __device__ __forceinline__ int count(int w) const {
        int n = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) n += max(0, min(32 * V, K - (j * nt + w * 32) * V));
        return n;
    }
};

// Waits for the stage that is read next and refills the one that was read last. With VEC a thread's own copies
// are all it reads; otherwise all threads' copies must have come, and all must have left the last stage.
template <bool VEC, typename F>
__device__ __forceinline__ void ring_step(F refill) {
    if constexpr (VEC) {
        refill();
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(NORM_STAGES - 1) : "memory");
    } else {
        asm volatile("cp.async.wait_group %0;" ::"n"(NORM_STAGES - 2) : "memory");
        if (blockDim.x == 32) __syncwarp();
        else __syncthreads();
        refill();
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
}

// The mean square is taken about the warp's own mean and moved to the row's mean afterwards, so the R rows cost one
// barrier. (Both means are sums divided by their count to the last place, so a row of equal values has deviation 0, as
// in the kernel above. The rounding of the warp's mean enters the mean square squared, and times its distance from the
// row's mean.)
// 8192 x 7168 bf16: 49.5 us, 73 % of the copy rate (a block a row, the kernel above: 62), RMS 41 us, 87 %; fp32 81 us,
// 88 %. What is left in bf16 is latency at few warps: 14 warps an SM issue in half of the cycles. (8 columns a thread,
// twice the warps, are there for rows of up to 256; on long rows they were tried in the backward pass only.)
template <typename XT, typename WT, int N, int R, int COLS>
__global__ void __launch_bounds__(NORM_RING_THREADS) layer_norm_ring_kernel(const __grid_constant__ NormParams p) {
    using Cols = NormColumns<XT, N, COLS>;
    constexpr bool VEC = Cols::VEC;
    extern __shared__ __align__(16) unsigned char s_norm[];
    __shared__ float2 s_red[2][R][32];
    pdl_launch_dependents();
    pdl_wait();
    const int K = p.K, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, nw = nt >> 5;
    const int step = gridDim.x * blockDim.y;
    const size_t total = static_cast<size_t>(p.T) * K;
    const int pitch = Cols::pitch(K);
    const Cols cols(K);
    const XT *x = static_cast<const XT *>(p.x);
    XT *ring = reinterpret_cast<XT *>(s_norm) + static_cast<size_t>(threadIdx.y) * NORM_STAGES * R * pitch;
    constexpr bool KEEP = N <= 16;   // w and b in registers, or read again (from L1) for every row
    Pair w[N / 2], b[N / 2];
    const auto parameters = [&] {
        if (p.w) {
            cols.load(static_cast<const WT *>(p.w), w);
        } else {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) w[e] = pair(1.f, 1.f);
        }
        if (p.b) {
            cols.load(static_cast<const WT *>(p.b), b);
        } else {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) b[e] = pair(0.f, 0.f);
        }
    };
    if constexpr (KEEP) parameters();
    const int count = cols.count(tid >> 5), count_of_lane = lane < nw ? cols.count(lane) : 0;
    const float own = static_cast<float>(count), inv_count = count ? 1.f / own : 0.f;
    const float fk = static_cast<float>(K), inv_k = 1.f / fk;
    const auto fetch = [&](int first, int stage) {
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (first + q * step < p.T)
                cols.fetch(ring + (stage * R + q) * pitch, x, static_cast<size_t>(first + q * step) * K, total);
    };
    int row = blockIdx.x * blockDim.y + threadIdx.y;   // T <= 2^30: no sum below overflows
#pragma unroll
    for (int s = 0; s + 1 < NORM_STAGES; ++s) {
        fetch(row + s * R * step, s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    for (int n = 0; row < p.T; ++n, row += R * step) {
        ring_step<VEC>([&] { fetch(row + (NORM_STAGES - 1) * R * step, stage == 0 ? NORM_STAGES - 1 : stage - 1); });
        Pair f[R][N / 2];
        float mu[R], m2[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mu[q] = m2[q] = 0.f;
            const size_t at = static_cast<size_t>(row + q * step) * K;
            if (row + q * step < p.T) {
                cols.load(ring + (stage * R + q) * pitch + cols.offset(at), f[q]);
                if (!p.rms) {
                    Pair s = f[q][0];
#pragma unroll
                    for (int e = 1; e < N / 2; ++e) s = s + f[q][e];
                    const float2 h = halves(s);
                    mu[q] = h.x + h.y;
                }
            }
        }
        stage = stage + 1 == NORM_STAGES ? 0 : stage + 1;
        if (!p.rms) {   // the warp's means
            if constexpr (R == 2) {
                const float2 s = warp_sum2(mu[0], mu[1]);
                mu[0] = mean_of(s.x, own, inv_count);
                mu[1] = mean_of(s.y, own, inv_count);
            } else {
                mu[0] = mean_of(warp_sum(mu[0]), own, inv_count);
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (row + q * step < p.T) m2[q] = cols.squares(f[q], mu[q]);
        if constexpr (R == 2) {
            const float2 s = warp_sum2(m2[0], m2[1]);
            m2[0] = s.x;
            m2[1] = s.y;
        } else {
            m2[0] = warp_sum(m2[0]);
        }
        if (nt > 32) {
            const int q_of = R == 2 && lane ? 1 : 0;
            if (lane < R) s_red[n & 1][lane][tid >> 5] = make_float2(q_of ? mu[R - 1] : mu[0], q_of ? m2[R - 1] : m2[0]);
            __syncthreads();   // the other half of s_red is free: all have left the last rows' sums
            const float c = static_cast<float>(count_of_lane);
            float2 v[R];
            float a[R];
#pragma unroll
            for (int q = 0; q < R; ++q) {
                v[q] = lane < nw ? s_red[n & 1][q][lane] : make_float2(0.f, 0.f);
                a[q] = v[q].x * c;
            }
            if (!p.rms) {
                const float2 s = R == 2 ? warp_sum2(a[0], a[R - 1]) : make_float2(warp_sum(a[0]), 0.f);
                mu[0] = mean_of(s.x, fk, inv_k);
                if (R == 2) mu[R - 1] = mean_of(s.y, fk, inv_k);
            }
#pragma unroll
            for (int q = 0; q < R; ++q) a[q] = p.rms ? v[q].y : fmaf(c * (v[q].x - mu[q]), v[q].x - mu[q], v[q].y);
            const float2 s = R == 2 ? warp_sum2(a[0], a[R - 1]) : make_float2(warp_sum(a[0]), 0.f);
            m2[0] = s.x;
            if (R == 2) m2[R - 1] = s.y;
        }
        if constexpr (!KEEP) parameters();
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int t = row + q * step;
            if (t >= p.T) break;   // the same for the whole team
            const float r = rsqrtf(fmaf(m2[q], inv_k, p.eps));   // within 2 ulp, as in the kernel above
            if (tid == 0) {
                if (p.mean) p.mean[t] = mu[q];
                if (p.rstd) p.rstd[t] = r;
            }
            const Pair c = pair(-mu[q], -mu[q]), rr = pair(r, r);
#pragma unroll
            for (int e = 0; e < N / 2; ++e) f[q][e] = fma2((f[q][e] + c) * rr, w[e], b[e]);
            if (p.y) cols.store(static_cast<XT *>(p.y) + static_cast<size_t>(t) * K, f[q]);
            if constexpr (VEC) {
                if (p.q) {   // K % 128 == 0: the threads of a slice are all inside the row or all outside
                    constexpr int V = Cols::V;
#pragma unroll
                    for (int j = 0; j < Cols::VPT; ++j) {
                        float v[V], m = 0.f;
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) {
                            const float2 h = halves(f[q][j * (V / 2) + e]);
                            v[2 * e] = h.x;
                            v[2 * e + 1] = h.y;
                            m = fmaxf(m, fmaxf(fabsf(h.x), fabsf(h.y)));
                        }
                        norm_cast<V>(p, v, m, t, j * nt + tid, K / V);
                    }
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
    float len, inv_len;         // K and 1/K: operands from here cost the row kernel no registers
};

// Long rows: dx of one row per blockDim.x threads, laid out as in the forward kernel.
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

// Rows too long for the kernel below (their ring does not fit): the column sums over one part of the rows.
// Block (32, 8), a thread a column, 8 rows at a time;
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

// dx, and the sums of dw and db, in one pass over dy and x: HBM-bound (three tensors of T·K). Teams, columns
// and the ring are those of the forward kernel, with rows of x and dy side by side; a thread's columns' dw
// and db stay in registers to the end (one running fp32 sum over the rows of a team: 56 of 8192), and R rows cost one
// barrier for their sums of u and u·(x - mu).
// dx = (dy·r)·w - r·c1 - xh·(r·c2) with c1 = mean(u), c2 = r·mean(u·(x - mu)). c1 is divided to the last place: where
// all u of a row are equal it has to cancel them, and an ulp left over would be multiplied by r.
// The teams' sums meet in shared memory and go to part[blockIdx.x] in a fixed order.
// 8192 x 7168 bf16, with the parts' sum: 70 us, 77 % of the copy rate; fp32 123 us, 88 %. A dx kernel and a column kernel
// took 250 us. 8 columns a thread (twice the threads, half the registers) spill: 127 to 142 us.
template <typename XT, typename WT, int N, int R, int COLS>
__global__ void __launch_bounds__(NORM_RING_THREADS) layer_norm_backward_kernel(const __grid_constant__ NormBackParams p) {
    using Cols = NormColumns<XT, N, COLS>;
    constexpr bool VEC = Cols::VEC;
    constexpr int H = N / 2;
    extern __shared__ __align__(16) unsigned char s_norm[];
    __shared__ float4 s_red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int K = p.K, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, teams = blockDim.y;
    const int step = gridDim.x * teams;
    const size_t total = static_cast<size_t>(p.T) * K;
    const int pitch = Cols::pitch(K);
    const Cols cols(K);
    const XT *x = static_cast<const XT *>(p.x), *dy = static_cast<const XT *>(p.dy);
    XT *ring = reinterpret_cast<XT *>(s_norm) + static_cast<size_t>(threadIdx.y) * NORM_STAGES * R * 2 * pitch;
    const Pair zero = pair(0.f, 0.f);
    constexpr bool KEEP = N <= 16;   // w in registers, or read again (from L1) for every row
    constexpr bool HOLD = R == 1 && N <= 16;   // the row stays in registers across its sums
    Pair w[H], aw[H], ab[H];
    const auto parameters = [&] {
        if (p.w) {
            cols.load(static_cast<const WT *>(p.w), w);
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) w[e] = pair(1.f, 1.f);
        }
    };
    if constexpr (KEEP) parameters();
#pragma unroll
    for (int e = 0; e < H; ++e) aw[e] = ab[e] = zero;
    const auto fetch = [&](int first, int stage) {
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (first + q * step < p.T) {
                const size_t at = static_cast<size_t>(first + q * step) * K;
                cols.fetch(ring + (stage * R + q) * 2 * pitch, x, at, total);
                cols.fetch(ring + ((stage * R + q) * 2 + 1) * pitch, dy, at, total);
            }
    };
    int row = blockIdx.x * teams + threadIdx.y;   // T <= 2^30: no sum below overflows
#pragma unroll
    for (int s = 0; s + 1 < NORM_STAGES; ++s) {
        fetch(row + s * R * step, s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // mean and rstd of the team's next 32 rows, one a lane: a load for each step's rows, prefetched a step ahead, was
    // waited for together with reads of the ring (85 us instead of 69 for 8192 x 7168, by the compiler's choice)
    float mean32, rstd32;
    const auto statistics = [&](int first) {
        const int at = first + lane * step;
        rstd32 = at < p.T ? p.rstd[at] : 0.f;
        mean32 = at < p.T && p.mean ? p.mean[at] : 0.f;
    };
    statistics(row);
    int stage = 0;
    for (int n = 0; row < p.T; ++n, row += R * step) {
        ring_step<VEC>([&] { fetch(row + (NORM_STAGES - 1) * R * step, stage == 0 ? NORM_STAGES - 1 : stage - 1); });
        if (n > 0 && n * R % 32 == 0) statistics(row);
        float mu[R], r[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mu[q] = __shfl_sync(0xFFFFFFFFu, mean32, (n * R + q) & 31);
            r[q] = __shfl_sync(0xFFFFFFFFu, rstd32, (n * R + q) & 31);
        }
        float sums[2 * R];
        Pair hx[HOLD ? H : 1], hd[HOLD ? H : 1];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            sums[2 * q] = sums[2 * q + 1] = 0.f;
            if (row + q * step < p.T) {
                const int off = cols.offset(static_cast<size_t>(row + q * step) * K);
                Pair fx[H], fd[H];
                if constexpr (!KEEP) parameters();
                cols.load(ring + (stage * R + q) * 2 * pitch + off, fx);
                cols.load(ring + ((stage * R + q) * 2 + 1) * pitch + off, fd);
                if constexpr (HOLD) {
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        hx[e] = fx[e];
                        hd[e] = fd[e];
                    }
                }
                const Pair c = pair(-mu[q], -mu[q]);
                Pair s1 = zero, s2 = zero;
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const Pair u = fd[e] * w[e];
                    s1 = s1 + u;
                    s2 = fma2(u, fx[e] + c, s2);
                }
                const float2 h1 = halves(s1), h2 = halves(s2);
                sums[2 * q] = h1.x + h1.y;
                sums[2 * q + 1] = h2.x + h2.y;
            }
        }
        float means[2 * R];   // of u and of u·(x - mu)
        if constexpr (R == 2) {
            float s = warp_sum4_spread(make_float4(sums[0], sums[1], sums[2], sums[3]));
            if (nt > 32) {
                if (lane % 8 == 0) reinterpret_cast<float *>(&s_red[n & 1][tid >> 5])[lane / 8] = s;
                __syncthreads();   // the other half of s_red is free: all have left the last rows' sums
                s = warp_sum4_spread(lane < nt / 32 ? s_red[n & 1][lane] : make_float4(0.f, 0.f, 0.f, 0.f));
            }
            s = mean_of(s, p.len, p.inv_len);
#pragma unroll
            for (int i = 0; i < 4; ++i) means[i] = __shfl_sync(0xFFFFFFFFu, s, 8 * i);
        } else {
            float2 s = warp_sum2(sums[0], sums[1]);
            if (nt > 32) {
                if (lane == 0) s_red[n & 1][tid >> 5] = make_float4(s.x, s.y, 0.f, 0.f);
                __syncthreads();
                const float4 v = lane < nt / 32 ? s_red[n & 1][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                s = warp_sum2(v.x, v.y);
            }
            // mean_of, written out: the call's order of instructions costs odd rows 5 % (8192 x 4097 120 us, so 115)
            means[0] = fmaf(fmaf(-(s.x * p.inv_len), p.len, s.x), p.inv_len, s.x * p.inv_len);
            means[1] = s.y * p.inv_len;
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (row + q * step < p.T) {
                const size_t at = static_cast<size_t>(row + q * step) * K;
                Pair fx[H], fd[H];   // two rows are read again: they would not fit across the sums
                if constexpr (!KEEP) parameters();
                if constexpr (HOLD) {
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        fx[e] = hx[e];
                        fd[e] = hd[e];
                    }
                } else {
                    cols.load(ring + (stage * R + q) * 2 * pitch + cols.offset(at), fx);
                    cols.load(ring + ((stage * R + q) * 2 + 1) * pitch + cols.offset(at), fd);
                }
                const float rq = r[q], b0 = p.mean ? -rq * means[2 * q] : 0.f;
                const float a0 = -rq * (rq * means[2 * q + 1]);   // -r·c2, c2 = r·mean(u·d)
                const Pair c = pair(-mu[q], -mu[q]), rr = pair(rq, rq), pa = pair(a0, a0), pb = pair(b0, b0);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const Pair xh = (fx[e] + c) * rr;
                    ab[e] = ab[e] + fd[e];
                    aw[e] = fma2(fd[e], xh, aw[e]);
                    fx[e] = fma2(fd[e] * rr, w[e], fma2(xh, pa, pb));
                }
                cols.store(static_cast<XT *>(p.dx) + at, fx);
            }
        }
        stage = stage + 1 == NORM_STAGES ? 0 : stage + 1;
    }
    if (!p.part) return;
    float *part = p.part + static_cast<size_t>(blockIdx.x) * 2 * K;
    float *out = teams == 1 ? part : reinterpret_cast<float *>(s_norm) + threadIdx.y * 2 * K;
    if (teams > 1) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();   // the ring becomes the teams' sums [teams][2][K]
    }
    cols.store(out, aw);
    cols.store(out + K, ab);
    if (teams == 1) return;
    __syncthreads();
    for (int i = threadIdx.y * nt + tid; i < 2 * K; i += teams * nt) {
        float a = 0.f;
        for (int m = 0; m < teams; ++m) a += reinterpret_cast<const float *>(s_norm)[m * 2 * K + i];
        part[i] = a;
    }
}

// dw and db from the parts: block (32, 16), a column a thread; thread row y adds the parts y, y + 16, ...,
// and the 16 sums are added in their order. Grid (ceil(K/32), 2).
__global__ void __launch_bounds__(512) layer_norm_parts_kernel(const __grid_constant__ NormBackParams p) {
    __shared__ float s_sum[16][33];
    pdl_launch_dependents();
    pdl_wait();
    const int col = blockIdx.x * 32 + threadIdx.x;
    float *out = blockIdx.y ? p.db : p.dw;
    float a = 0.f;
    if (out && col < p.K) {
        const float *part = p.part + static_cast<size_t>(blockIdx.y) * p.K + col;
#pragma unroll 8
        for (int i = threadIdx.y; i < p.parts; i += 16) a += part[static_cast<size_t>(i) * 2 * p.K];
    }
    s_sum[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && out && col < p.K) {
#pragma unroll
        for (int i = 1; i < 16; ++i) a += s_sum[i][threadIdx.x];
        out[col] = a;
    }
}

}  // namespace dg
