/*
 * dg.h — C ABI of the B200 (sm_100a) FP8 block-scaled NT GEMM library.
 *
 * The operation is D = C + A·Bᵀ in NT layout: A is [M,K] and B is [N,K], both K-contiguous
 * e4m3 (OCP E4M3FN). A carries one fp32 scale per 1×128 K-slice of each row, B one fp32
 * scale per 128×128 block, and C and D are bf16. Sources: the DeepGEMM write-ups —
 * likun.im/craft/deepgemm §一 (the D = C + A·Bᵀ NT convention; dense, M-grouped contiguous
 * and masked GEMMs) and §二 (the register_apis list: fp8_gemm_nt, m_grouped_*_contiguous with
 * grouped_layout, m_grouped_*_masked with masked_m / expected_m, transform_sf);
 * aitangshan.cn/news/1491278 技术原理 §4 (block-wise scaling, one scale per block, applied
 * after the multiplication); likun.im §五 (the LHS scales need a TMA-aligned, transposed
 * layout).
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller. The library neither frees
 *    nor keeps them after the call returns; the memory must stay valid until the work queued
 *    on `stream` has finished.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream). Every
 *    call is asynchronous with respect to the host and never synchronises the device.
 *  - Kb = K/128 and Nb = ceil(N/128). "pad4(x)" is x rounded up to a multiple of 4, so that
 *    every row of an MN-major fp32 scale array starts on a 16-byte boundary
 *    (dg_sf_ld(x) returns it).
 *  - Layout of the A scales ("sfa"): fp32 [Kb][pad4(M)], MN-major: sfa[kb*pad4(M) + m]
 *    scales A[m, kb*128 .. kb*128+127]. Entries m >= M are padding and never read.
 *  - Layout of the B scales ("sfb"): fp32 [G][Nb][Kb]: sfb[(g*Nb + nb)*Kb + kb] scales
 *    B[g, nb*128 .. nb*128+127, kb*128 .. kb*128+127] (G = 1 for the dense GEMM).
 *  - Argument errors are reported synchronously, before anything is queued:
 *      DG_ERR_INVALID_ARG (a size out of range, a NULL where a tensor is required),
 *      DG_ERR_ALIGNMENT (a base pointer not 16-byte aligned),
 *      DG_ERR_UNSUPPORTED (no device of compute capability 10.0 current).
 *    A failed launch returns DG_ERR_CUDA. Faults that only the device can see (an expert id
 *    in grouped_layout >= G, masked_m[g] > M_max, a pipeline wait that ran out of time) set a
 *    per-device error word that dg_get_device_error() returns. Nothing aborts the process
 *    and nothing throws across this ABI.
 *  - Preconditions of the GEMMs: K % 128 == 0, N % 8 == 0 (16-byte D rows), M >= 0.
 *    The results of the GEMMs satisfy |D - ref| <= 2^-7·|ref| + 1e-2·rms(ref) against the
 *    exact fp64 value of the same block-scaled operands. Every GEMM is deterministic: the
 *    same inputs give the same bits, call after call.
 *  - Environment variables, each read once per process:
 *      DG_WAIT_TIMEOUT_MS  the limit of every pipeline wait inside a kernel (default 4000);
 *                          on expiry the kernel stops and DG_ERR_TIMEOUT is reported.
 *    For experiments and tests only (they change which kernel runs, never the result beyond
 *    the stated bound): DG_FORCE_PAIR=0|1 (CTA pairs for the tile GEMM), DG_FORCE_BN=128|256,
 *    DG_FORCE_SWAP=0|1 (few-row kernels off for M <= 128, or on for the masked layout),
 *    DG_FEW_ROW=streamk|cluster, DG_SPLITK_S=1|2|3|4|6|8|16 (cluster size), DG_ONE_ISSUER=1
 *    (one MMA-issuing thread per CTA instead of two), DG_TAIL_SPLIT=0|2..64 (the dense tile
 *    GEMM's last-wave split off, or S pieces per last-wave tile). Debug only:
 *    DG_TEST_SKIP_RELEASE=1|2|3|4 makes one kernel withhold barrier arrives or partial flags,
 *    so that a wait runs out of time (failure tests).
 */
#ifndef DG_H
#define DG_H

#include <stdint.h>

#if defined(__GNUC__)
#define DG_API __attribute__((visibility("default")))
#else
#define DG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dg_status {
    DG_OK = 0,
    DG_ERR_INVALID_ARG = 1,
    DG_ERR_ALIGNMENT = 2,
    DG_ERR_UNSUPPORTED = 3,
    DG_ERR_CUDA = 4,
    DG_ERR_TIMEOUT = 5,
    DG_ERR_DEVICE = 6
} dg_status;

/* Dense FP8 NT GEMM, D = C + A·Bᵀ (likun.im/craft/deepgemm §二, fp8_gemm_nt).
 *   a   e4m3 [M,K] row-major;          sfa fp32 [Kb][pad4(M)]
 *   b   e4m3 [N,K] row-major;          sfb fp32 [Nb][Kb]
 *   c   bf16 [M,N] row-major or NULL (then C = 0); may alias d
 *   d   bf16 [M,N] row-major, written in full.
 * M may be 0 (nothing is queued). For M <= 128 the K blocks are split over several SMs:
 *   - with few 128-column tiles (at most 64) and K <= 8192, over a thread-block cluster per
 *     tile, whose partial sums meet in distributed shared memory (no scratch at all);
 *   - otherwise over every SM (stream-K), whose partial sums meet in a library-owned
 *     workspace of the (device, stream) pair, allocated (cudaMalloc, sm_count x 128 KB plus
 *     the flags) by the pair's first call that wants it and kept until the process ends; a
 *     first call made under CUDA-graph capture cannot allocate and computes with the tile
 *     kernel instead.
 * For M > 128 (the persistent tile kernel), when the tiles do not fill a whole number of
 * waves of resident CTAs, the last wave's tiles are cut along K into pieces run at once on
 * otherwise idle SMs, whose partial sums meet in the same workspace (in a fixed order); without
 * a workspace (a first call under graph capture) the last wave runs whole.
 * Every choice gives the same result within the stated bound, and each is deterministic. */
DG_API dg_status dg_fp8_gemm_nt(const void *a, const float *sfa, const void *b, const float *sfb,
                         const void *c, void *d, int M, int N, int K, void *stream);

/* dg_fp8_gemm_nt's stream-K path for M <= 128 without any allocation, for callers that must
 * not call cudaMalloc (an allocator-owning runtime, a pre-planned memory arena, a decode loop
 * that must not add allocations). Same arguments, and the same result bit for bit as
 * dg_fp8_gemm_nt whenever that call takes the stream-K kernel (the same kernel and the same
 * split of the work), but the kernel's scratch (the fp32 partial sums, their flags and a launch
 * epoch) is a fixed static __device__ array of the library, 16 MB + 1 KB, instead of a
 * per-stream workspace; every GPU that loads the library holds it until the process exits.
 * The first call of any entry point on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call before any stream
 * capture. The array is shared by every call on a device and keeps what the last call left:
 * calls that overlap on the GPU (on different streams, or replays of captured graphs that run
 * at the same time) race on it and must not be made. Flags left by a launch that stopped early
 * (after DG_ERR_TIMEOUT) are never taken for a later launch's: each launch waits for its own
 * ticket. The pages have no counterpart of this entry point.
 * Errors: those of dg_fp8_gemm_nt, plus DG_ERR_UNSUPPORTED (nothing queued) when M > 128 or
 * when the device has more than 256 SMs (the array's capacity). */
DG_API dg_status dg_fp8_gemm_nt_noalloc(const void *a, const float *sfa, const void *b, const float *sfb,
                                        const void *c, void *d, int M, int N, int K, void *stream);

/* Dense FP8 NT GEMM with UE8M0 (power-of-two) scales, applied by the tensor core's
 * block-scaled MMA (likun.im §五: SM100 wants packed UE8M0 scales, four per 32-bit word; §二:
 * disable_ue8m0_cast). D = C + A·Bᵀ with the block scaling of dg_fp8_gemm_nt, every scale
 * being 2^(byte - 127):
 *   a   e4m3 [M,K];   sfa uint32 [ceil(Kb/4)][pad4(M)]: byte kb%4 of word (kb/4, m) scales
 *                     A[m, kb*128 .. kb*128+127]   (dg_cast_fp8_per_token_ue8m0 writes it)
 *   b   e4m3 [N,K];   sfb uint32 [Nb][ceil(Kb/4)]: byte kb%4 of word (nb, kb/4) scales the
 *                     128x128 block (nb, kb) of B   (dg_cast_fp8_per_block_ue8m0 writes it)
 *   c   bf16 [M,N] or NULL (may alias d);   d  bf16 [M,N].
 * Since every sfa·sfb is a power of two the hardware applies it exactly and accumulates all K
 * blocks in TMEM (fp32). Extra precondition: N % 16 == 0. Errors as for dg_fp8_gemm_nt. */
DG_API dg_status dg_fp8_gemm_nt_ue8m0(const void *a, const uint32_t *sfa, const void *b, const uint32_t *sfb,
                                      const void *c, void *d, int M, int N, int K, void *stream);

/* The dense GEMM in the other three storage layouts the pages name (likun.im §一,
 * "fp8_fp4_gemm_{nt,nn,tn,tt}"; §二, "同类: _nn / _tn / _tt"). The first letter is A's
 * storage, the second B's: A "n" = [M,K] (K contiguous), A "t" = [K,M] (M contiguous);
 * B "t" = [N,K] (K contiguous), B "n" = [K,N] (N contiguous). The product is the NT one,
 * D[m,n] = C[m,n] + sum_k A_log[m,k]·B_log[n,k], with the same scales:
 *   sfa fp32 [Kb][pad4(M)] (one per row m and 128-wide K slice), sfb fp32 [Nb][Kb] (one per
 *   128x128 block of B_log), c/d bf16 [M,N] row-major as for dg_fp8_gemm_nt.
 *   nn: a [M,K], b [K,N];   tn: a [K,M], b [K,N];   tt: a [K,M], b [N,K].
 * An MN-major operand reaches the tensor core through MN-major shared-memory descriptors, with
 * no transpose pass. Extra precondition: M % 16 == 0 when A is MN-major and N % 16 == 0 when B
 * is (16-byte rows for the tensor-map loads), else DG_ERR_INVALID_ARG. Every M takes the tile
 * kernel (no few-row split). Errors as for dg_fp8_gemm_nt. */
DG_API dg_status dg_fp8_gemm_nn(const void *a, const float *sfa, const void *b, const float *sfb,
                                const void *c, void *d, int M, int N, int K, void *stream);
DG_API dg_status dg_fp8_gemm_tn(const void *a, const float *sfa, const void *b, const float *sfb,
                                const void *c, void *d, int M, int N, int K, void *stream);
DG_API dg_status dg_fp8_gemm_tt(const void *a, const float *sfa, const void *b, const float *sfb,
                                const void *c, void *d, int M, int N, int K, void *stream);

/* K-grouped FP8 GEMM for the MoE weight gradient (likun.im §一, "沿 K 轴分组的
 * k_grouped_fp8_gemm_tn（MoE 反向）"; §二, k_grouped_fp8_gemm_tn_contiguous with ks_cpu and
 * recipe (1,1,128)). The K dimension (tokens) of both operands is cut into G consecutive groups
 * of ks[g] tokens; group g gives D[g] = C[g] + A_gᵀ·B_g:
 *   a   e4m3 [sum_K, M] (token-major, M contiguous: the "T" operand)
 *   sfa fp32 [sum_K/128][pad4(M)]: one scale per channel m per 128 tokens
 *   b   e4m3 [sum_K, N] (token-major, N contiguous: the "N" operand)
 *   sfb fp32 [sum_K/128][pad4(N)]: one scale per channel n per 128 tokens
 *   c   fp32 [G, M, N] or NULL (C = 0); may alias d.   d  fp32 [G, M, N], written in full.
 *   ks         host array [G] of the group sizes, each a multiple of 128 (0 allowed: D[g] = C[g])
 *   ks_device  the same G values in device memory (int32), read by the kernel.
 * D[g,m,n] = C[g,m,n] + sum_{kb in g} sfa[kb][m]·sfb[kb][n]·sum_{k in kb} A[k,m]·B[k,n].
 * Preconditions: 1 <= G <= 511, M % 16 == 0, N % 16 == 0, 16-byte aligned pointers. A device
 * value that is not a multiple of 128 or reaches past the host's sum sets the device error word
 * (DG_ERR_DEVICE) and its group is computed as empty. */
DG_API dg_status dg_k_grouped_fp8_gemm_tn_contiguous(const void *a, const float *sfa, const void *b,
                                                     const float *sfb, const float *c, float *d,
                                                     const int *ks, const int32_t *ks_device, int G,
                                                     int M, int N, void *stream);

/* M-grouped "contiguous" FP8 NT GEMM for MoE prefill (likun.im §二,
 * m_grouped_*_gemm_nt_contiguous; zwt0204.github.io "DeepGEMM deep dive", the grouped-layout
 * constraint). The rows of A are the tokens of all G experts stacked, each expert's block
 * padded to a multiple of 128 rows.
 *   a   e4m3 [M_sum,K];                sfa fp32 [Kb][M_sum]   (M_sum % 128 == 0)
 *   b   e4m3 [G,N,K];                  sfb fp32 [G][Nb][Kb]
 *   grouped_layout  int32 [M_sum] on the device: the expert id of each row, -1 for a
 *       padding row. Every aligned 128-row block belongs to one expert; the block's expert is
 *       read from its first row. A block whose first row is -1 is skipped.
 *   c   bf16 [M_sum,N] or NULL;        d bf16 [M_sum,N].
 * D rows of padding rows have no defined value (they may be written). An id >= G sets the
 * device error word and its block is skipped. */
DG_API dg_status dg_m_grouped_fp8_gemm_nt_contiguous(const void *a, const float *sfa, const void *b,
                                              const float *sfb, const void *c, void *d,
                                              const int32_t *grouped_layout, int M_sum, int N,
                                              int K, int G, void *stream);

/* M-grouped "masked" FP8 NT GEMM for MoE decode (likun.im §二, m_grouped_*_gemm_nt_masked;
 * §四: it consumes the low-latency dispatch output). Expert g owns rows [0, masked_m[g]) of
 * its [M_max,K] slice of A.
 *   a   e4m3 [G,M_max,K];              sfa fp32 [G][Kb][pad4(M_max)]
 *   b   e4m3 [G,N,K];                  sfb fp32 [G][Nb][Kb]
 *   masked_m  int32 [G] on the device, read by the kernel (values > M_max are clamped to
 *       M_max and set the device error word; negative values count as 0).
 *   expected_m  host-side hint of the typical masked_m, used only to choose tile shapes:
 *       128-row tiles when expected_m <= 128, 256-row CTA-pair tiles above (0 = use M_max).
 *   c   bf16 [G,M_max,N] or NULL;      d bf16 [G,M_max,N].
 * Rows r >= masked_m[g] of D are never written and their A rows never reach D. */
DG_API dg_status dg_m_grouped_fp8_gemm_nt_masked(const void *a, const float *sfa, const void *b,
                                          const float *sfb, const void *c, void *d,
                                          const int32_t *masked_m, int expected_m, int G,
                                          int M_max, int N, int K, void *stream);

/* Scale-layout transform (likun.im §二 transform_sf / get_mn_major_tma_aligned_tensor; §五:
 * LHS scales in a TMA-aligned transposed layout).
 *   sf_kmajor  fp32 [batch][MN][Kb] (one row of Kb scales per token)
 *   sf_mnmajor fp32 [batch][Kb][pad4(MN)]; the pad4 tail of every row is written with 0.
 * The two buffers must not overlap. */
DG_API dg_status dg_transform_sf(const float *sf_kmajor, float *sf_mnmajor, int batch, int MN, int Kb,
                          void *stream);

/* Per-token FP8 cast of activations (block-wise scaling, aitangshan.cn 技术原理 §4, at
 * 1×128 granularity). For every row m and K-slice kb: amax = max|x|, s = amax/448 (s = 1 when
 * amax = 0), q = e4m3(x/s) rounded to nearest-even and saturated to ±448.
 *   x   bf16 [batch,M,K];  q e4m3 [batch,M,K];  sfa fp32 [batch][Kb][pad4(M)] (padding
 *   entries are not written). K % 128 == 0. */
DG_API dg_status dg_cast_fp8_per_token(const void *x, void *q, float *sfa, int batch, int M, int K,
                                void *stream);

/* Per-block FP8 cast of weights, 128×128 blocks (same rule; a partial last block of rows
 * uses its valid rows only).
 *   x   bf16 [batch,N,K];  q e4m3 [batch,N,K];  sfb fp32 [batch][Nb][Kb]. K % 128 == 0. */
DG_API dg_status dg_cast_fp8_per_block(const void *x, void *q, float *sfb, int batch, int N, int K,
                                void *stream);

/* The per-token cast written straight into the M-grouped contiguous layout: the MoE dispatch
 * in front of dg_m_grouped_fp8_gemm_nt_contiguous (likun.im §二, m_grouped_*_contiguous with
 * grouped_layout; the pages' "fused cast + grouped GEMM"). Token t of x is quantised as by
 * dg_cast_fp8_per_token and written to row dst_rows[t] of q and sfa, in one pass, and the
 * GEMM that follows on the stream overlaps its prologue with this kernel (programmatic
 * dependent launch, as every kernel of the library).
 *   x         bf16 [T,K] (tokens in any order)
 *   dst_rows  int32 [T] on the device: the token's row in the contiguous layout, -1 to drop it;
 *             no two tokens may share a row. A row >= M_sum sets the device error word
 *             (DG_ERR_DEVICE) and the token is dropped.
 *   q         e4m3 [M_sum,K];  sfa fp32 [Kb][pad4(M_sum)] (the GEMM's layouts). Rows no token
 *             maps to (the padding of each expert's block) are not written.
 * K % 128 == 0. */
DG_API dg_status dg_cast_fp8_per_token_scatter(const void *x, const int32_t *dst_rows, void *q, float *sfa, int T,
                                               int M_sum, int K, void *stream);

/* Per-token and per-block FP8 casts with UE8M0 scales (likun.im §五: on SM100 the scales are
 * packed UE8M0, four per 32-bit word; §二: disable_ue8m0_cast). The scale of a block is the
 * smallest power of two s = 2^e >= amax/448 (the fp32 quotient), e clamped to [-127, 127]
 * (s = 1 when amax = 0), kept as the byte e + 127; q = e4m3(x/s) as for the fp32 casts (the
 * division by a power of two is exact). Scales are packed four K blocks per uint32 word, K
 * block kb in bits 8·(kb%4) .. 8·(kb%4)+7; bytes of K blocks >= Kb hold 127.
 *   per token: x bf16 [batch,M,K]; q e4m3 [batch,M,K];
 *              sfa uint32 [batch][ceil(Kb/4)][pad4(M)] (MN-major; padding entries m >= M
 *              are not written)
 *   per block: x bf16 [batch,N,K]; q e4m3 [batch,N,K]; sfb uint32 [batch][Nb][ceil(Kb/4)]
 * K % 128 == 0. */
DG_API dg_status dg_cast_fp8_per_token_ue8m0(const void *x, void *q, uint32_t *sfa, int batch, int M, int K,
                                             void *stream);
DG_API dg_status dg_cast_fp8_per_block_ue8m0(const void *x, void *q, uint32_t *sfb, int batch, int N, int K,
                                             void *stream);

/* Per-channel FP8 cast along the token dimension, the recipe (1,1,128) of the K-grouped GEMM's
 * operands (likun.im §二, k_grouped_fp8_gemm_tn_contiguous): for every 128-token block tb and
 * channel c, amax = max_t |x[t,c]| over the block's tokens, s = amax/448 (s = 1 when amax = 0),
 * q[t,c] = e4m3(x[t,c]/s), nearest-even, saturated to ±448 (the per-token cast's rule).
 *   x   bf16 [T,C] token-major;  q e4m3 [T,C];  sf fp32 [T/128][pad4(C)] (padding entries are
 *   not written). T % 128 == 0, C % 8 == 0, else DG_ERR_INVALID_ARG. */
DG_API dg_status dg_cast_fp8_per_channel(const void *x, void *q, float *sf, int T, int C, void *stream);

/* Element types of the operators below that take more than one. Their row counts T are at most 2^30; outputs
 * may overlap inputs only where it is said. */
typedef enum dg_dtype { DG_BF16 = 0, DG_FP32 = 1 } dg_dtype;

/* Layer norm (rms = 0) or RMS norm (rms != 0) over the K elements of each row, with the
 * per-token FP8 cast of the result as an option (the pages fuse such casts into the producing
 * kernel; likun.im §五 gives the scales' layout):
 *   mu = mean(x) (0 for rms), r = 1/sqrt(mean((x-mu)^2) + eps), y = (x-mu)·r·weight + bias.
 *   x       [T,K] of x_type (DG_BF16 or DG_FP32)
 *   weight, bias  [K] of w_type, or NULL (ones, zeros); rms takes no bias
 *   y       [T,K] of x_type, or NULL when only the codes are wanted; may be x itself
 *   q, sfa  e4m3 [T,K] and fp32 [Kb][pad4(T)] by the rule of dg_cast_fp8_per_token, or both NULL;
 *           the cast is of the fp32 y before its rounding to x_type; padding entries of sfa are
 *           not written. Needs K % 128 == 0.
 *   mean, rstd  fp32 [T], what dg_layer_norm_backward reads, or NULL.
 * Any K from 1 to 32768, eps >= 0. Statistics are fp32. */
DG_API dg_status dg_layer_norm(const void *x, const void *weight, const void *bias, void *y, void *q, float *sfa,
                               float *mean, float *rstd, int T, int K, float eps, int rms, int x_type, int w_type,
                               void *stream);

/* Gradients of dg_layer_norm's y, with xh = (x-mean)·rstd and u = dy·weight:
 *   dx = rstd·(u - mean_K(u) - xh·mean_K(u·xh))  (mean = NULL, the RMS form: without mean_K(u));
 *   dw = sum over rows of dy·xh, db = sum over rows of dy: fp32 [K], either may be NULL. With
 *   T = 0 they are zeroed.
 *   dy, x, dx  [T,K] of x_type; weight [K] of w_type or NULL; mean, rstd as the forward wrote them.
 *   workspace  dg_layer_norm_backward_workspace(T, K) bytes of device memory, 16-byte aligned, for
 *              this call alone until its work on the stream is done; NULL when dw and db are.
 * dx may not overlap dy or x. The sums over rows are taken in a fixed order. */
DG_API dg_status dg_layer_norm_backward(const void *dy, const void *x, const void *weight, const float *mean,
                                        const float *rstd, void *dx, float *dw, float *db, void *workspace,
                                        long long workspace_bytes, int T, int K, int x_type, int w_type, void *stream);
DG_API long long dg_layer_norm_backward_workspace(int T, int K);

/* Routing of tokens to experts, in front of the grouped GEMMs. For a token with logits x[E]:
 *   s = softmax(x) or sigmoid(x); choice values c = s + bias (bias may be NULL);
 *   the E experts form `groups` groups of E/groups; a group's value is the sum of its group_top
 *   (1 or 2) largest c, and the topk_groups groups of largest value are kept;
 *   ids = the k experts of largest c in the kept groups, in falling order of c;
 *   w_j = s[ids_j], divided by their sum if renorm, times scale. The bias is in no weight.
 * Equal values are taken in the order of their index. The choice is that of the 64-bit values: scores
 * that differ by less than an fp32 rounding are not confused (without a bias the logits are compared, which holds where
 * 64-bit scores are equal, too). A logit of -inf or a bias of -inf
 * takes the expert out of the choice; so does a NaN, which also sets the device error word; a
 * logit of +inf counts as the largest finite fp32. Where fewer than k experts are left, the last
 * ids are -1 and their weights 0. A group with fewer than group_top experts left counts those
 * it has.
 *   logits  [T,E] of dtype (DG_BF16 or DG_FP32);  bias fp32 [E] or NULL
 *   ids     int32 [T,k];  weights fp32 [T,k]
 * Limits: E <= 1024, k <= min(E, 32), groups <= 32 and E % groups == 0. */
typedef enum dg_score { DG_SCORE_SOFTMAX = 0, DG_SCORE_SIGMOID = 1 } dg_score;
DG_API dg_status dg_moe_route(const void *logits, const float *bias, int32_t *ids, float *weights, int T, int E, int k,
                              int groups, int topk_groups, int group_top, int score, int renorm, float scale, int dtype,
                              void *stream);

/* Gradient of the logits from the gradient of dg_moe_route's weights (fp32 [T,k]). ids are the
 * forward's; -1 (any negative id) has no gradient, an id >= E sets the device error word and is
 * left out, an id that stands twice in a row gets both gradients. grad_logits [T,E] of dtype is
 * written in full; it may not overlap logits. score, renorm and scale are the forward's. */
DG_API dg_status dg_moe_route_backward(const float *grad_weights, const void *logits, const int32_t *ids,
                                       void *grad_logits, int T, int E, int k, int score, int renorm, float scale,
                                       int dtype, void *stream);

/* Rows of the grouped layouts for the expert ids of T tokens (int32 [T,k]; ids outside [0,G),
 * such as -1 or another rank's experts, are dropped: row -1). Rows follow the order of the pairs
 * (token, then place), so they are the same in every run.
 *   contiguous: expert g's rows start where the earlier experts' rows, each padded to a multiple
 *     of 128, end. dst_rows int32 [T,k]; grouped_layout int32 [M_sum] as
 *     dg_m_grouped_fp8_gemm_nt_contiguous reads it (-1 for padding and all rows behind the last
 *     expert); ks int32 [G], the padded row counts (ks_device of the K-grouped GEMM), or NULL.
 *     M_sum % 128 == 0; T·k + 127·min(G, T·k), rounded up to a multiple of 128, fits any ids.
 *   masked: expert g's rows are g·M_max, g·M_max + 1, ...; masked_m int32 [G], their number.
 * A pair whose row would lie outside M_sum (or at or behind M_max) gets row -1 and sets the device
 * error word; ks and masked_m are clamped.
 * Limits: G <= 1024, T·k <= 2^30, G·M_max < 2^31. */
DG_API dg_status dg_moe_layout_contiguous(const int32_t *ids, int32_t *dst_rows, int32_t *grouped_layout, int32_t *ks,
                                          int T, int k, int G, int M_sum, void *stream);
DG_API dg_status dg_moe_layout_masked(const int32_t *ids, int32_t *dst_rows, int32_t *masked_m, int T, int k, int G,
                                      int M_max, void *stream);

/* dg_cast_fp8_per_token_scatter for k rows per token and both grouped layouts: token t is
 * quantised once and written to the rows dst_rows[t][0..k-1] (int32 [T,k]; negative: none) of G
 * groups of M rows:
 *   contiguous: G = 1, M = M_sum;   masked: G experts of M = M_max rows
 *   q e4m3 [G·M,K];  sfa fp32 [G][Kb][pad4(M)]. Rows no token maps to are not written.
 * No two pairs may share a row. A row >= G·M sets the device error word and is left out.
 * K % 128 == 0, G·M < 2^31, T·k <= 2^30. */
DG_API dg_status dg_cast_fp8_per_token_scatter_topk(const void *x, const int32_t *dst_rows, void *q, float *sfa, int T,
                                                    int k, int G, int M, int K, void *stream);

/* The experts' results back to the tokens: y[t] = c[t] + sum_j weights[t,j]·d[dst_rows[t,j]].
 *   d  bf16 [R,N] (R = M_sum, or G·M_max);  dst_rows int32 [T,k] (negative: left out; its row is
 *   not read);  weights fp32 [T,k] or NULL (ones: also the gradient of the dispatch);
 *   c  bf16 [T,N] or NULL (may be y);  y bf16 [T,N]. Sums are fp32 in the order of j, rounded once.
 * N % 8 == 0, k <= 32. A row >= R sets the device error word and is left out. */
DG_API dg_status dg_moe_combine(const void *d, const int32_t *dst_rows, const float *weights, const void *c, void *y,
                                int T, int k, int N, int R, void *stream);

/* Gradients of dg_moe_combine: grad_d[dst_rows[t,j]] = weights[t,j]·grad_y[t] (bf16 [R,N]) and
 * grad_weights[t,j] = <grad_y[t], d[dst_rows[t,j]]> (fp32 [T,k], 0 for a negative row). Either may be
 * NULL; d is read for grad_weights only. (The gradient of c is grad_y.) No two pairs may share a
 * row. Rows of grad_d that no pair maps to are not written, except that with grouped_layout
 * (int32 [R] or NULL) the rows whose entry is negative are zeroed, as the K-grouped weight
 * gradient wants its padding. grad_d may not overlap d. */
DG_API dg_status dg_moe_combine_backward(const void *grad_y, const void *d, const int32_t *dst_rows,
                                         const float *weights, const int32_t *grouped_layout, void *grad_d,
                                         float *grad_weights, int T, int k, int N, int R, void *stream);

/* pad4(mn): the leading dimension of an MN-major scale array. */
DG_API int dg_sf_ld(int mn);

/* Waits for `stream`, then returns and clears the current device's error word
 * (DG_OK, DG_ERR_TIMEOUT or DG_ERR_DEVICE). */
DG_API dg_status dg_get_device_error(void *stream);

/* Static, human-readable name of a status code. */
DG_API const char *dg_status_string(dg_status status);

/* Name of the GEMM kernel that the calling thread's last GEMM call launched ("" before the
 * first): "gemm_kernel", "gemm_kernel (CTA pairs)", "gemm_kernel (last-wave split S)" or
 * "gemm_kernel (CTA pairs, last-wave split S)" when the last wave's tiles were cut into S K
 * pieces, "gemm_swap_kernel (stream-K)",
 * "gemm_splitk_kernel (cluster split-K)" or "gemm_bs_kernel (UE8M0 block-scaled MMA)". For
 * benchmarks and profiles; valid until the thread's next GEMM call. */
DG_API const char *dg_last_kernel(void);

/* Number of kernels the calling thread's last launching GEMM call launched (0 before the
 * first): 1, or 2 for a tile GEMM whose last-wave split ran behind a launch of the whole
 * waves. For benchmarks that count launches. */
DG_API int dg_last_launch_count(void);

/* Bytes of device memory the library has allocated with cudaMalloc so far, over all devices
 * (the few-row stream-K workspaces); the static arrays of the module are not counted. */
DG_API long long dg_allocated_bytes(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_H */
