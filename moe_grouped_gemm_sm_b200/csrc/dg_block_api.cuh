// dg_block_api.cuh — the C ABI of the operators around the experts' products: argument checks, launch
// shapes and launches. Part of dg_api.cu (it uses that file's device facts and launch helper).
#pragma once
#include "dg_norm.cuh"
#include "dg_route.cuh"
#include "dg_rows.cuh"

namespace {

constexpr int kNormMaxK = 32768;
constexpr int kNormLongParts = 64;    // row parts of the dw / db sums of long rows
constexpr int kNormSms = 148;         // the SMs that rings are cut for, not those of the current device: the backward
                                      // pass's workspace is asked for before there need be one
constexpr int kNormRing = 200 << 10;  // bytes of shared memory for the ring of rows

constexpr int kMaxRows = 1 << 30;

bool valid_type(int t) { return t == DG_BF16 || t == DG_FP32; }

// f(vector size, vectors per thread, grid, block) of the register kernel, the first two as compile-time constants: one
// warp a row, 8 rows a block, for rows of up to 4 vectors a lane; else a block a row. Few rows (fewer than two
// blocks per SM) spread a row over as many threads as it has vectors; many rows keep 4 vectors in flight per
// thread. Rows that are not whole 16-byte vectors go element by element (V = 1, 4 or 32 a thread).
template <typename XT, typename F>
dg_status norm_dispatch(int T, int K, int sm_count, F f) {
    constexpr int VMAX = 16 / static_cast<int>(sizeof(XT));
    using std::integral_constant;
    const int v = K % VMAX == 0 ? VMAX : 1, nv = K / v;
    int vpt = T < 2 * sm_count ? 1 : 4;
    dim3 block(32, 8, 1), grid(static_cast<unsigned>((T + 7) / 8), 1, 1);
    if (nv <= 128) {
        vpt = nv <= 32 ? 1 : (nv <= 64 ? 2 : 4);
    } else {
        while ((nv + vpt - 1) / vpt > dg::NORM_MAX_THREADS) vpt *= 2;
        block = dim3(static_cast<unsigned>(((nv + vpt - 1) / vpt + 31) / 32 * 32), 1, 1);
        grid = dim3(static_cast<unsigned>(T), 1, 1);
    }
    if (v == 1) {
        if (vpt <= 4) return f(integral_constant<int, 1>(), integral_constant<int, 4>(), grid, block);
        return f(integral_constant<int, 1>(), integral_constant<int, 32>(), grid, block);
    }
    if (vpt == 1) return f(integral_constant<int, VMAX>(), integral_constant<int, 1>(), grid, block);
    if (vpt == 2) return f(integral_constant<int, VMAX>(), integral_constant<int, 2>(), grid, block);
    if constexpr (VMAX == 4)   // fp32 rows of more than 16384
        if (vpt == 8) return f(integral_constant<int, VMAX>(), integral_constant<int, 8>(), grid, block);
    return f(integral_constant<int, VMAX>(), integral_constant<int, 4>(), grid, block);
}

// Launch shape of the ring kernels (`tensors` rows side by side: 1 forward, 2 backward): 16 columns a thread, 8 for
// rows of up to 256, 32 for rows of more than 8192, 16 single ones where rows are not whole vectors; two rows per
// step where the ring holds them. Warps as teams for rows of one warp; otherwise a block a row, and as many
// blocks per SM as 512 threads and the rings allow. blocks = 0: the row is too long.
struct NormRingShape {
    int cols, n, r, threads, teams, blocks;
    size_t smem;
};

NormRingShape norm_ring_shape(int T, int K, int x_type, int tensors) {
    const int size = x_type == DG_BF16 ? 2 : 4, c = 16 / size;
    NormRingShape s{};
    s.cols = K % c == 0 ? dg::COLS_VECTORS : dg::COLS_SINGLE;
    s.n = s.cols && K <= 256 ? 8 : (K <= 16 * dg::NORM_RING_THREADS ? 16 : 32);
    s.threads = ((K + s.n - 1) / s.n + 31) / 32 * 32;
    s.teams = s.threads == 32 ? 4 : 1;
    if (s.cols && K == s.n * s.threads) s.cols = dg::COLS_EXACT;
    const size_t row = static_cast<size_t>(dg::NORM_STAGES) * tensors * (s.cols ? K : (K + 2 * c - 2) / c * c) * size;
    // Two rows a step where the rings of the blocks that the threads allow still fit an SM (8192 x 4096 fp32 backward
    // takes 86 us with one block of two rows an SM and 71 with two of one row). Backward, a single row stays in registers
    // between its sums and dx, and that beats two rows unless the columns are exact: 8192 x 7168 bf16 68 us by two and 72
    // by one, 8192 x 1000 24 and 19, 8192 x 3001 73 and 62.
    const int most = std::max(1, dg::NORM_RING_THREADS / (s.threads * s.teams));
    const size_t ring = static_cast<size_t>(kNormRing), sm = static_cast<size_t>(220 << 10);
    s.r = s.n <= 16 && 2 * row * s.teams * most <= sm && 2 * row <= ring ? 2 : 1;
    if (tensors == 2 && s.n == 16 && s.cols != dg::COLS_EXACT) s.r = 1;
    if (s.threads > dg::NORM_RING_THREADS || (s.n == 32 && !s.cols) || s.r * row > ring) return s;
    s.smem = s.teams * s.r * row;
    const int per_sm = std::max(1, std::min(most, static_cast<int>(sm / s.smem)));
    s.blocks = std::min((T + s.teams - 1) / s.teams, kNormSms * per_sm);
    // Backward: two rows a block at least, once every SM has a block; its part of dw and db is as long as a row
    // (1000 x 1024 bf16 10.0 us, one row a block 11.4; 2000 x 1001 fp32 15.8 and 18.3; four rows 8.3 and 20.8).
    if (tensors == 2) s.blocks = std::min(s.blocks, std::max(kNormSms, T / s.teams / 2));
    return s;
}

// A kernel with a ring: more than 48 KB of shared memory, the kernel's static part included, has to be
// allowed once per device.
template <typename P>
dg_status launch_norm_ring(void (*kernel)(P), std::atomic<int> *ready, const P &p, const NormRingShape &s, cudaStream_t st) {
    if (s.smem > (40 << 10)) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return DG_ERR_CUDA;
        if (!ready[dev].load()) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRing) != cudaSuccess)
                return DG_ERR_CUDA;
            ready[dev].store(1);
        }
    }
    Launch ln(dim3(static_cast<unsigned>(s.blocks), 1, 1),
              dim3(static_cast<unsigned>(s.threads), static_cast<unsigned>(s.teams), 1), s.smem, st);
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, kernel, p));
}

template <typename XT, typename WT, int N, int R, int COLS>
dg_status launch_layer_norm_ring(const dg::NormParams &p, const NormRingShape &s, cudaStream_t st) {
    static std::atomic<int> ready[kMaxDevices];
    return launch_norm_ring<dg::NormParams>(dg::layer_norm_ring_kernel<XT, WT, N, R, COLS>, ready, p, s, st);
}

template <typename XT, typename WT>
dg_status run_layer_norm(const dg::NormParams &p, int x_type, int sm_count, cudaStream_t st) {
    // Rows of up to 128 stay with the register kernel: 200000 x 128 bf16 takes 45 us there and 56 us here;
    // 65536 x 512 takes 33 us there and 24 us here.
    if (p.T >= 2 * kNormSms && p.K > 128) {
        const NormRingShape s = norm_ring_shape(p.T, p.K, x_type, 1);
        if (s.blocks) {
            if (s.n == 32)
                return s.cols == dg::COLS_EXACT ? launch_layer_norm_ring<XT, WT, 32, 1, dg::COLS_EXACT>(p, s, st)
                                                : launch_layer_norm_ring<XT, WT, 32, 1, dg::COLS_VECTORS>(p, s, st);
            if (s.n == 8)
                return s.cols == dg::COLS_EXACT ? launch_layer_norm_ring<XT, WT, 8, 2, dg::COLS_EXACT>(p, s, st)
                                                : launch_layer_norm_ring<XT, WT, 8, 2, dg::COLS_VECTORS>(p, s, st);
            if (s.r == 2)
                return s.cols == dg::COLS_EXACT     ? launch_layer_norm_ring<XT, WT, 16, 2, dg::COLS_EXACT>(p, s, st)
                       : s.cols == dg::COLS_VECTORS ? launch_layer_norm_ring<XT, WT, 16, 2, dg::COLS_VECTORS>(p, s, st)
                                                    : launch_layer_norm_ring<XT, WT, 16, 2, dg::COLS_SINGLE>(p, s, st);
        }
    }
    return norm_dispatch<XT>(p.T, p.K, sm_count, [&](auto v, auto vpt, dim3 grid, dim3 block) {
        Launch ln(grid, block, 0, st);
        return from_cuda(cudaLaunchKernelEx(
            &ln.cfg, dg::layer_norm_kernel<XT, WT, decltype(v)::value, decltype(vpt)::value>, p));
    });
}

int norm_parts(int T, int K, int x_type) {
    const NormRingShape s = norm_ring_shape(T, K, x_type, 2);
    return s.blocks ? s.blocks : std::max(1, std::min(kNormLongParts, (T + 7) / 8));
}

template <typename XT, typename WT, int N, int R, int COLS>
dg_status launch_norm_backward(const dg::NormBackParams &p, const NormRingShape &s, cudaStream_t st) {
    static std::atomic<int> ready[kMaxDevices];
    return launch_norm_ring<dg::NormBackParams>(dg::layer_norm_backward_kernel<XT, WT, N, R, COLS>, ready, p, s, st);
}

// Rows too long for the ring (bf16 above 16384, fp32 above 8533, single columns above 8192): dx by a block a row,
// 8 or 16 vectors or 64 elements a thread, then the column sums.
template <typename XT, typename WT, int V, int VPT>
dg_status launch_norm_long(const dg::NormBackParams &p, cudaStream_t st) {
    const int nt = ((p.K / V + VPT - 1) / VPT + 31) / 32 * 32;
    Launch ln(dim3(static_cast<unsigned>(p.T), 1, 1), dim3(static_cast<unsigned>(nt), 1, 1), 0, st);
    const dg_status s = from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::layer_norm_dx_kernel<XT, WT, V, VPT>, p));
    if (s != DG_OK || !p.part) return s;
    Launch sums(dim3(static_cast<unsigned>((p.K + 31) / 32), static_cast<unsigned>(p.parts), 1), dim3(32, 8, 1), 0, st);
    return from_cuda(cudaLaunchKernelEx(&sums.cfg, dg::layer_norm_dwdb_kernel<XT>, p));
}

template <typename XT, typename WT>
dg_status run_layer_norm_backward(dg::NormBackParams p, int x_type, cudaStream_t st) {
    const NormRingShape sh = norm_ring_shape(p.T, p.K, x_type, 2);
    p.parts = norm_parts(p.T, p.K, x_type);
    if (!p.dw && !p.db) p.part = nullptr;
    dg_status s;
    if (sh.blocks) {
        if (sh.n == 32)
            s = sh.cols == dg::COLS_EXACT ? launch_norm_backward<XT, WT, 32, 1, dg::COLS_EXACT>(p, sh, st)
                                          : launch_norm_backward<XT, WT, 32, 1, dg::COLS_VECTORS>(p, sh, st);
        else if (sh.n == 8)
            s = sh.cols == dg::COLS_EXACT ? launch_norm_backward<XT, WT, 8, 2, dg::COLS_EXACT>(p, sh, st)
                                          : launch_norm_backward<XT, WT, 8, 2, dg::COLS_VECTORS>(p, sh, st);
        else if (sh.cols == dg::COLS_EXACT)
            s = sh.r == 2 ? launch_norm_backward<XT, WT, 16, 2, dg::COLS_EXACT>(p, sh, st)
                          : launch_norm_backward<XT, WT, 16, 1, dg::COLS_EXACT>(p, sh, st);
        else if (sh.cols == dg::COLS_VECTORS)
            s = launch_norm_backward<XT, WT, 16, 1, dg::COLS_VECTORS>(p, sh, st);
        else
            s = launch_norm_backward<XT, WT, 16, 1, dg::COLS_SINGLE>(p, sh, st);
    } else {
        constexpr int V = 16 / static_cast<int>(sizeof(XT));
        if (p.K % V != 0)
            s = launch_norm_long<XT, WT, 1, 64>(p, st);
        else if (p.K <= V * 8 * dg::NORM_DX_MAX_THREADS)
            s = launch_norm_long<XT, WT, V, 8>(p, st);
        else if constexpr (V == 4)
            s = launch_norm_long<XT, WT, V, 16>(p, st);
        else
            s = DG_ERR_INVALID_ARG;   // no bf16 row is longer than 8·8·512
    }
    if (s != DG_OK || !p.part) return s;
    Launch ln(dim3(static_cast<unsigned>((p.K + 31) / 32), 2, 1), dim3(32, 16, 1), 0, st);
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::layer_norm_parts_kernel, p));
}

// Argument checks that both directions of the routing share.
dg_status check_route(int T, int E, int k, int score, int dtype) {
    if (T < 0 || T > kMaxRows || E <= 0 || E > dg::ROUTE_MAX_E || k <= 0 || k > dg::ROUTE_MAX_K || k > E ||
        !valid_type(dtype) || (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID))
        return DG_ERR_INVALID_ARG;
    return DG_OK;
}

// A warp takes a token; the warps of ROUTE_BLOCKS blocks an SM take further ones (they keep the bias in registers).
template <typename LT>
dg_status run_route(const dg::RouteParams &p, int sm_count, cudaStream_t st) {
    const int blocks = std::min((p.T + dg::ROUTE_WARPS - 1) / dg::ROUTE_WARPS, sm_count * dg::ROUTE_BLOCKS);
    Launch ln(dim3(static_cast<unsigned>(blocks), 1, 1), dim3(32 * dg::ROUTE_WARPS, 1, 1), 0, st);
    const int per_lane = (p.E + 31) / 32;
    if (per_lane <= 1) return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::route_kernel<LT, 1>, p));
    if (per_lane <= 2) return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::route_kernel<LT, 2>, p));
    if (per_lane <= 4) return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::route_kernel<LT, 4>, p));
    if (per_lane <= 8) return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::route_kernel<LT, 8>, p));
    if (per_lane <= 16) return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::route_kernel<LT, 16>, p));
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::route_kernel<LT, 32>, p));
}

bool layout_sizes_ok(int T, int k, int G) {
    return T >= 0 && k > 0 && G > 0 && G <= dg::LAYOUT_MAX_G && static_cast<long long>(T) * k <= (1LL << 30);
}

// 2^BITS >= G. The counts of [warps][G] stay within 48 KB of shared memory; a second block of the cluster comes with
// more than 64 pairs a warp (its barriers cost about as much as two rounds of 32 pairs). Clusters of 16 where
// the device can hold one, else of 8.
template <bool MASKED, int BITS>
dg_status launch_layout(dg::LayoutParams p, cudaStream_t st) {
    const auto kernel = dg::layout_kernel<MASKED, BITS>;
    const int warps = p.G <= 256 ? 32 : (p.G <= 512 ? 16 : 8);
    const size_t smem = static_cast<size_t>(p.G) * 4 * (3 + warps);
    static std::atomic<int> most[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return DG_ERR_CUDA;
    if (most[dev].load() == 0) {
        int n = 0;
        Launch ln(dim3(16, 1, 1), dim3(1024, 1, 1), 46 << 10, st, 16);   // the most that any G takes: 11·4·1024
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &ln.cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        most[dev].store(n > 0 ? 16 : 8);
    }
    int blocks = 1;
    while (blocks < most[dev].load() && p.n > blocks * warps * 64) blocks *= 2;
    const int all = blocks * warps;
    p.per_warp = static_cast<int>(std::max(1LL, (static_cast<long long>(p.n) + all * 32 - 1) / (all * 32))) * 32;
    Launch ln(dim3(static_cast<unsigned>(blocks), 1, 1), dim3(static_cast<unsigned>(32 * warps), 1, 1), smem, st, blocks);
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, kernel, p));
}

template <bool MASKED>
dg_status run_layout(const int32_t *ids, int32_t *dst_rows, int32_t *grouped_layout, int32_t *counts, int T, int k, int G,
                     int M, cudaStream_t st) {
    const DeviceInfo *di = nullptr;
    dg_status s = device_info(&di);
    if (s != DG_OK) return s;
    dg::LayoutParams p{};
    p.ids = ids;
    p.dst_rows = dst_rows;
    p.grouped_layout = grouped_layout;
    p.counts = counts;
    p.err = di->err;
    p.n = T * k;
    p.G = G;
    p.M = M;
    if (G <= 32) return launch_layout<MASKED, 5>(p, st);
    if (G <= 256) return launch_layout<MASKED, 8>(p, st);
    return launch_layout<MASKED, 10>(p, st);
}

}  // namespace

extern "C" {

dg_status dg_layer_norm(const void *x, const void *weight, const void *bias, void *y, void *q, float *sfa, float *mean,
                        float *rstd, int T, int K, float eps, int rms, int x_type, int w_type, void *stream) {
    if (!x || (!y && !q) || (q != nullptr) != (sfa != nullptr) || T < 0 || T > kMaxRows || K <= 0 || K > kNormMaxK ||
        !(eps >= 0.f) ||
        !valid_type(x_type) || !valid_type(w_type) || (rms && bias) || (q && K % 128 != 0))
        return DG_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(weight) || !aligned16(bias) || !aligned16(y) || !aligned16(q) || !aligned16(sfa))
        return DG_ERR_ALIGNMENT;
    if (T == 0) return DG_OK;
    const DeviceInfo *di = nullptr;
    dg_status s = device_info(&di);
    if (s != DG_OK) return s;
    dg::NormParams p{};
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.y = y;
    p.q = static_cast<uint8_t *>(q);
    p.sfa = sfa;
    p.mean = mean;
    p.rstd = rstd;
    p.T = T;
    p.K = K;
    p.ld = pad4(T);
    p.rms = rms ? 1 : 0;
    p.eps = eps;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x_type == DG_BF16)
        return w_type == DG_BF16 ? run_layer_norm<__nv_bfloat16, __nv_bfloat16>(p, x_type, di->sm_count, st)
                                 : run_layer_norm<__nv_bfloat16, float>(p, x_type, di->sm_count, st);
    return w_type == DG_BF16 ? run_layer_norm<float, __nv_bfloat16>(p, x_type, di->sm_count, st)
                             : run_layer_norm<float, float>(p, x_type, di->sm_count, st);
}

long long dg_layer_norm_backward_workspace(int T, int K) {
    if (T <= 0 || T > kMaxRows || K <= 0 || K > kNormMaxK) return 0;
    return static_cast<long long>(std::max(norm_parts(T, K, DG_BF16), norm_parts(T, K, DG_FP32))) * 2 * K * 4;
}

dg_status dg_layer_norm_backward(const void *dy, const void *x, const void *weight, const float *mean, const float *rstd,
                                 void *dx, float *dw, float *db, void *workspace, long long workspace_bytes, int T, int K,
                                 int x_type, int w_type, void *stream) {
    if (!dy || !x || !rstd || !dx || T < 0 || T > kMaxRows || K <= 0 || K > kNormMaxK || !valid_type(x_type) ||
        !valid_type(w_type))
        return DG_ERR_INVALID_ARG;
    if ((dw || db) && T > 0 && (!workspace || workspace_bytes < dg_layer_norm_backward_workspace(T, K)))
        return DG_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(weight) || !aligned16(dx) || !aligned16(dw) || !aligned16(db) ||
        !aligned16(workspace))
        return DG_ERR_ALIGNMENT;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // sums over no rows
        if ((dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(K) * 4, st) != cudaSuccess) ||
            (db && cudaMemsetAsync(db, 0, static_cast<size_t>(K) * 4, st) != cudaSuccess))
            return DG_ERR_CUDA;
        return DG_OK;
    }
    const DeviceInfo *di = nullptr;
    dg_status s = device_info(&di);
    if (s != DG_OK) return s;
    dg::NormBackParams p{};
    p.dy = dy;
    p.x = x;
    p.w = weight;
    p.mean = mean;
    p.rstd = rstd;
    p.dx = dx;
    p.part = static_cast<float *>(workspace);
    p.dw = dw;
    p.db = db;
    p.T = T;
    p.K = K;
    p.len = static_cast<float>(K);
    p.inv_len = 1.f / p.len;
    if (x_type == DG_BF16)
        return w_type == DG_BF16 ? run_layer_norm_backward<__nv_bfloat16, __nv_bfloat16>(p, x_type, st)
                                 : run_layer_norm_backward<__nv_bfloat16, float>(p, x_type, st);
    return w_type == DG_BF16 ? run_layer_norm_backward<float, __nv_bfloat16>(p, x_type, st)
                             : run_layer_norm_backward<float, float>(p, x_type, st);
}

dg_status dg_moe_route(const void *logits, const float *bias, int32_t *ids, float *weights, int T, int E, int k,
                       int groups, int topk_groups, int group_top, int score, int renorm, float scale, int dtype,
                       void *stream) {
    if (!logits || !ids || !weights) return DG_ERR_INVALID_ARG;
    dg_status s = check_route(T, E, k, score, dtype);
    if (s != DG_OK) return s;
    if (groups <= 0 || groups > dg::ROUTE_MAX_GROUPS || E % groups != 0 || topk_groups <= 0 || topk_groups > groups ||
        group_top < 1 || group_top > 2 || !(scale - scale == 0.f))
        return DG_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights)) return DG_ERR_ALIGNMENT;
    if (T == 0) return DG_OK;
    const DeviceInfo *di = nullptr;
    s = device_info(&di);
    if (s != DG_OK) return s;
    dg::RouteParams p{};
    p.logits = logits;
    p.bias = bias;
    p.ids = ids;
    p.weights = weights;
    p.err = di->err;
    p.T = T;
    p.E = E;
    p.k = k;
    p.groups = topk_groups == groups ? 1 : groups;   // every group kept: no choice between groups
    p.topk_groups = topk_groups;
    p.group_size = E / p.groups;
    p.rows_per_group = p.group_size % 32 == 0 ? p.group_size / 32 : 0;
    p.group_top = group_top;
    p.score = score;
    p.renorm = renorm ? 1 : 0;
    p.scale = scale;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == DG_BF16 ? run_route<__nv_bfloat16>(p, di->sm_count, st) : run_route<float>(p, di->sm_count, st);
}

dg_status dg_moe_route_backward(const float *grad_weights, const void *logits, const int32_t *ids, void *grad_logits,
                                int T, int E, int k, int score, int renorm, float scale, int dtype, void *stream) {
    if (!grad_weights || !logits || !ids || !grad_logits || !(scale - scale == 0.f)) return DG_ERR_INVALID_ARG;
    dg_status s = check_route(T, E, k, score, dtype);
    if (s != DG_OK) return s;
    if (!aligned16(grad_weights) || !aligned16(logits) || !aligned16(ids) || !aligned16(grad_logits))
        return DG_ERR_ALIGNMENT;
    if (T == 0) return DG_OK;
    const DeviceInfo *di = nullptr;
    s = device_info(&di);
    if (s != DG_OK) return s;
    dg::RouteParams p{};
    p.logits = logits;
    p.ids = const_cast<int32_t *>(ids);
    p.grad_w = grad_weights;
    p.grad_logits = grad_logits;
    p.err = di->err;
    p.T = T;
    p.E = E;
    p.k = k;
    p.score = score;
    p.renorm = renorm ? 1 : 0;
    p.scale = scale;
    Launch ln(dim3(static_cast<unsigned>((T + dg::ROUTE_WARPS - 1) / dg::ROUTE_WARPS), 1, 1),
              dim3(32 * dg::ROUTE_WARPS, 1, 1), 0, static_cast<cudaStream_t>(stream));
    return from_cuda(dtype == DG_BF16 ? cudaLaunchKernelEx(&ln.cfg, dg::route_backward_kernel<__nv_bfloat16>, p)
                                      : cudaLaunchKernelEx(&ln.cfg, dg::route_backward_kernel<float>, p));
}

dg_status dg_moe_layout_contiguous(const int32_t *ids, int32_t *dst_rows, int32_t *grouped_layout, int32_t *ks, int T, int k,
                                   int G, int M_sum, void *stream) {
    if ((T > 0 && (!ids || !dst_rows)) || (M_sum > 0 && !grouped_layout) || !layout_sizes_ok(T, k, G) || M_sum < 0 ||
        M_sum % 128 != 0)
        return DG_ERR_INVALID_ARG;
    if (!aligned16(ids) || !aligned16(dst_rows) || !aligned16(grouped_layout) || !aligned16(ks)) return DG_ERR_ALIGNMENT;
    return run_layout<false>(ids, dst_rows, grouped_layout, ks, T, k, G, M_sum, static_cast<cudaStream_t>(stream));
}

dg_status dg_moe_layout_masked(const int32_t *ids, int32_t *dst_rows, int32_t *masked_m, int T, int k, int G, int M_max,
                               void *stream) {
    if ((T > 0 && (!ids || !dst_rows)) || !masked_m || !layout_sizes_ok(T, k, G) || M_max < 0 ||
        static_cast<long long>(G) * M_max >= (1LL << 31))
        return DG_ERR_INVALID_ARG;
    if (!aligned16(ids) || !aligned16(dst_rows) || !aligned16(masked_m)) return DG_ERR_ALIGNMENT;
    return run_layout<true>(ids, dst_rows, nullptr, masked_m, T, k, G, M_max, static_cast<cudaStream_t>(stream));
}

dg_status dg_cast_fp8_per_token_scatter_topk(const void *x, const int32_t *dst_rows, void *q, float *sfa, int T, int k,
                                             int G, int M, int K, void *stream) {
    if (!x || !dst_rows || !q || !sfa || T < 0 || k <= 0 || G <= 0 || M < 0 || K <= 0 || K % 128 != 0 ||
        static_cast<long long>(G) * M >= (1LL << 31) || static_cast<long long>(T) * k > (1LL << 30))
        return DG_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(q) || !aligned16(sfa)) return DG_ERR_ALIGNMENT;
    if (T == 0 || M == 0) return DG_OK;
    const DeviceInfo *di = nullptr;
    dg_status s = device_info(&di);
    if (s != DG_OK) return s;
    // a thread takes 16 elements; few tokens are cut along K until there are two blocks per SM
    int threads = std::min(dg::SCATTER_THREADS, (K / 16 + 31) / 32 * 32);
    while (static_cast<long long>(T) * ((K / 16 + threads - 1) / threads) < 2LL * di->sm_count && threads > 64)
        threads = (threads / 2 + 31) / 32 * 32;
    const int parts = T < 2 * di->sm_count ? (K / 16 + threads - 1) / threads : 1;
    if (parts > 65535) return DG_ERR_INVALID_ARG;
    Launch ln(dim3(static_cast<unsigned>(T), static_cast<unsigned>(parts), 1), dim3(static_cast<unsigned>(threads), 1, 1), 0,
              static_cast<cudaStream_t>(stream));
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::cast_scatter_topk_kernel, static_cast<const __nv_bfloat16 *>(x),
                                        dst_rows, static_cast<uint8_t *>(q), sfa, k, K, M, pad4(M),
                                        static_cast<long long>(G) * M, di->err));
}

dg_status dg_moe_combine(const void *d, const int32_t *dst_rows, const float *weights, const void *c, void *y, int T,
                         int k, int N, int R, void *stream) {
    if ((R > 0 && !d) || (T > 0 && (!dst_rows || !y)) || T < 0 || T > kMaxRows || k <= 0 ||
        k > dg::COMBINE_MAX_K || N <= 0 || N % 8 != 0 || R < 0)
        return DG_ERR_INVALID_ARG;
    if (!aligned16(d) || !aligned16(c) || !aligned16(y)) return DG_ERR_ALIGNMENT;
    if (T == 0) return DG_OK;
    const DeviceInfo *di = nullptr;
    dg_status s = device_info(&di);
    if (s != DG_OK) return s;
    dg::CombineParams p{};
    p.d = static_cast<const __nv_bfloat16 *>(d);
    p.dst = dst_rows;
    p.w = weights;
    p.c = static_cast<const __nv_bfloat16 *>(c);
    p.y = static_cast<__nv_bfloat16 *>(y);
    p.err = di->err;
    p.T = T;
    p.k = k;
    p.N = N;
    p.R = R;
    const unsigned parts = static_cast<unsigned>(std::min(65535, (N / 8 + dg::COMBINE_THREADS - 1) / dg::COMBINE_THREADS));
    Launch ln(dim3(static_cast<unsigned>(T), parts, 1), dim3(dg::COMBINE_THREADS, 1, 1), 0,
              static_cast<cudaStream_t>(stream));
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::combine_kernel, p));
}

dg_status dg_moe_combine_backward(const void *grad_y, const void *d, const int32_t *dst_rows, const float *weights,
                                  const int32_t *grouped_layout, void *grad_d, float *grad_weights, int T, int k, int N,
                                  int R, void *stream) {
    if ((T > 0 && (!grad_y || !dst_rows)) || (T > 0 && R > 0 && !grad_d && !grad_weights) ||
        (R > 0 && grad_weights && !d) || (grouped_layout && !grad_d) || T < 0 || T > kMaxRows || k <= 0 ||
        k > dg::COMBINE_MAX_K || N <= 0 || N % 8 != 0 || R < 0)
        return DG_ERR_INVALID_ARG;
    if (!aligned16(grad_y) || !aligned16(d) || !aligned16(grad_d)) return DG_ERR_ALIGNMENT;
    const DeviceInfo *di = nullptr;
    dg_status s = device_info(&di);
    if (s != DG_OK) return s;
    dg::CombineParams p{};
    p.d = static_cast<const __nv_bfloat16 *>(d);
    p.dst = dst_rows;
    p.w = weights;
    p.gy = static_cast<const __nv_bfloat16 *>(grad_y);
    p.layout = grouped_layout;
    p.gd = static_cast<__nv_bfloat16 *>(grad_d);
    p.gw = grad_weights;
    p.err = di->err;
    p.T = T;
    p.k = k;
    p.N = N;
    p.R = R;
    const long long zero_blocks = grouped_layout ? std::min(R, 8 * di->sm_count) : 0;
    const long long blocks = T + zero_blocks;
    if (blocks == 0) return DG_OK;
    if (blocks >= (1LL << 31)) return DG_ERR_INVALID_ARG;
    Launch ln(dim3(static_cast<unsigned>(blocks), 1, 1), dim3(dg::COMBINE_THREADS, 1, 1), 0,
              static_cast<cudaStream_t>(stream));
    return from_cuda(cudaLaunchKernelEx(&ln.cfg, dg::combine_backward_kernel, p));
}

}  // extern "C"
