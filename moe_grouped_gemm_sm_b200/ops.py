"""torch-tensor conveniences over the C ABI: they allocate outputs with torch and pass
pointers. All arithmetic happens in libdg_b200.so.

Layouts (see include/dg.h): e4m3 tensors are torch.uint8 holding the codes; ``sfa`` is fp32
[batch?][Kb][pad4(M)] (MN-major), ``sfb`` fp32 [G?][ceil(N/128)][Kb]; C and D are bf16 (fp32 for
the K-grouped GEMM); UE8M0 scales are int32 words of four packed bytes.

Each function checks that its tensors are contiguous CUDA tensors, allocates what it returns
(or writes ``out``) and makes one C-ABI call on ``stream`` (default: the current stream).

The operators around the experts' products (``layer_norm*``, ``moe_*``, ``cast_per_token_scatter_topk``) also
check types and shapes and that all tensors are on one device; they run on that device, and
allocate their results and workspaces for the stream that they run on. Tensors start on 16 bytes; the
routing, its gradient and the layouts also take slices that do not, and copy them first. The gradients are
explicit functions; no autograd graph is built.
"""
from __future__ import annotations

import functools

import torch

from . import _lib


def _pad4(x: int) -> int:
    return (x + 3) // 4 * 4


def _check_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must live on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def cast_per_token(x: torch.Tensor, stream=None):
    """bf16 [M,K] or [batch,M,K] -> (e4m3 codes uint8 same shape, sfa fp32 [batch?][Kb][pad4(M)])."""
    _check_cuda(x)
    assert x.dtype == torch.bfloat16
    squeeze = x.dim() == 2
    xb = x.unsqueeze(0) if squeeze else x
    B, M, K = xb.shape
    q = torch.empty((B, M, K), dtype=torch.uint8, device=x.device)
    sfa = torch.zeros((B, K // 128, _pad4(M)), dtype=torch.float32, device=x.device)
    _lib.dg_cast_fp8_per_token(xb, q, sfa, B, M, K, stream)
    return (q[0], sfa[0]) if squeeze else (q, sfa)


def cast_per_block(w: torch.Tensor, stream=None):
    """bf16 [N,K] or [G,N,K] -> (e4m3 codes uint8 same shape, sfb fp32 [G?][ceil(N/128)][Kb])."""
    _check_cuda(w)
    assert w.dtype == torch.bfloat16
    squeeze = w.dim() == 2
    wb = w.unsqueeze(0) if squeeze else w
    G, N, K = wb.shape
    q = torch.empty((G, N, K), dtype=torch.uint8, device=w.device)
    sfb = torch.empty((G, (N + 127) // 128, K // 128), dtype=torch.float32, device=w.device)
    _lib.dg_cast_fp8_per_block(wb, q, sfb, G, N, K, stream)
    return (q[0], sfb[0]) if squeeze else (q, sfb)


def transform_sf(sf_kmajor: torch.Tensor, stream=None) -> torch.Tensor:
    """fp32 [MN,Kb] or [batch,MN,Kb] -> [Kb,pad4(MN)] or [batch,Kb,pad4(MN)]."""
    _check_cuda(sf_kmajor)
    squeeze = sf_kmajor.dim() == 2
    s = sf_kmajor.unsqueeze(0) if squeeze else sf_kmajor
    B, MN, Kb = s.shape
    out = torch.empty((B, Kb, _pad4(MN)), dtype=torch.float32, device=s.device)
    _lib.dg_transform_sf(s, out, B, MN, Kb, stream)
    return out[0] if squeeze else out


def fp8_gemm_nt(a, sfa, b, sfb, c=None, out=None, stream=None) -> torch.Tensor:
    """D = C + A·Bᵀ; a [M,K] codes, b [N,K] codes; returns bf16 [M,N]."""
    _check_cuda(a, sfa, b, sfb, c, out)
    M, K = a.shape
    N = b.shape[0]
    d = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _lib.dg_fp8_gemm_nt(a, sfa, b, sfb, c, d, M, N, K, stream)
    return d


def m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, grouped_layout, c=None, out=None, stream=None):
    """a [M_sum,K], b [G,N,K], grouped_layout int32 [M_sum]; returns bf16 [M_sum,N]."""
    _check_cuda(a, sfa, b, sfb, grouped_layout, c, out)
    M_sum, K = a.shape
    G, N, _ = b.shape
    d = out if out is not None else torch.empty((M_sum, N), dtype=torch.bfloat16, device=a.device)
    _lib.dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, c, d, grouped_layout, M_sum, N, K, G, stream)
    return d


def m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, masked_m, expected_m, c=None, out=None, stream=None):
    """a [G,M_max,K], b [G,N,K], masked_m int32 [G] (device); returns bf16 [G,M_max,N]
    (rows >= masked_m[g] keep whatever ``out`` held)."""
    _check_cuda(a, sfa, b, sfb, masked_m, c, out)
    G, M_max, K = a.shape
    N = b.shape[1]
    d = out if out is not None else torch.empty((G, M_max, N), dtype=torch.bfloat16, device=a.device)
    _lib.dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, c, d, masked_m, expected_m, G, M_max, N, K, stream)
    return d


def cast_per_token_scatter(x, dst_rows, M_sum, stream=None):
    """bf16 [T,K] tokens and int32 [T] destination rows (device) -> (e4m3 [M_sum,K], sfa fp32
    [Kb][pad4(M_sum)]) in the contiguous grouped layout; rows no token maps to stay zero."""
    _check_cuda(x, dst_rows)
    assert x.dtype == torch.bfloat16 and dst_rows.dtype == torch.int32
    T, K = x.shape
    q = torch.zeros((M_sum, K), dtype=torch.uint8, device=x.device)
    sfa = torch.zeros((K // 128, _pad4(M_sum)), dtype=torch.float32, device=x.device)
    _lib.dg_cast_fp8_per_token_scatter(x, dst_rows, q, sfa, T, M_sum, K, stream)
    return q, sfa


def cast_per_token_ue8m0(x, stream=None):
    """bf16 [M,K] -> (e4m3 [M,K], packed UE8M0 sfa int32 [ceil(Kb/4)][pad4(M)])."""
    _check_cuda(x)
    assert x.dtype == torch.bfloat16
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sfa = torch.zeros(((K // 128 + 3) // 4, _pad4(M)), dtype=torch.int32, device=x.device)
    _lib.dg_cast_fp8_per_token_ue8m0(x, q, sfa, 1, M, K, stream)
    return q, sfa


def cast_per_block_ue8m0(w, stream=None):
    """bf16 [N,K] -> (e4m3 [N,K], packed UE8M0 sfb int32 [ceil(N/128)][ceil(Kb/4)])."""
    _check_cuda(w)
    assert w.dtype == torch.bfloat16
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    sfb = torch.zeros(((N + 127) // 128, (K // 128 + 3) // 4), dtype=torch.int32, device=w.device)
    _lib.dg_cast_fp8_per_block_ue8m0(w, q, sfb, 1, N, K, stream)
    return q, sfb


def fp8_gemm_nt_ue8m0(a, sfa, b, sfb, c=None, out=None, stream=None) -> torch.Tensor:
    """D = C + A·Bᵀ with packed UE8M0 scales (cast_per_token_ue8m0 / cast_per_block_ue8m0)."""
    _check_cuda(a, sfa, b, sfb, c, out)
    M, K = a.shape
    N = b.shape[0]
    d = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _lib.dg_fp8_gemm_nt_ue8m0(a, sfa, b, sfb, c, d, M, N, K, stream)
    return d


def fp8_gemm(layout, a, sfa, b, sfb, c=None, out=None, stream=None) -> torch.Tensor:
    """The dense GEMM in layout "nt", "nn", "tn" or "tt" (A then B: "n" = K contiguous for A,
    "t" = M contiguous; for B "t" = [N,K], "n" = [K,N]); sfa fp32 [Kb][pad4(M)], sfb fp32
    [ceil(N/128)][Kb] for the logical operands; returns bf16 [M,N]."""
    _check_cuda(a, sfa, b, sfb, c, out)
    if layout not in ("nt", "nn", "tn", "tt"):
        raise ValueError(f"layout {layout!r}")
    K, M = (a.shape[0], a.shape[1]) if layout[0] == "t" else (a.shape[1], a.shape[0])
    N = b.shape[1] if layout[1] == "n" else b.shape[0]
    d = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    getattr(_lib, "dg_fp8_gemm_" + layout)(a, sfa, b, sfb, c, d, M, N, K, stream)
    return d


def cast_per_channel(x, stream=None):
    """bf16 [T,C] token-major (T % 128 == 0) -> (e4m3 [T,C], sf fp32 [T/128][pad4(C)])."""
    _check_cuda(x)
    assert x.dtype == torch.bfloat16
    T, C = x.shape
    q = torch.empty((T, C), dtype=torch.uint8, device=x.device)
    sf = torch.zeros((T // 128, _pad4(C)), dtype=torch.float32, device=x.device)
    _lib.dg_cast_fp8_per_channel(x, q, sf, T, C, stream)
    return q, sf


def k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, ks, c=None, out=None, stream=None) -> torch.Tensor:
    """a e4m3 [sum_K,M] and b e4m3 [sum_K,N] (token-major, from cast_per_channel), ks the G group
    sizes (host ints, multiples of 128); returns fp32 D [G,M,N] with D[g] = C[g] + A_gᵀ·B_g."""
    _check_cuda(a, sfa, b, sfb, c, out)
    ks = [int(k) for k in ks]
    M, N = a.shape[1], b.shape[1]
    ks_dev = torch.tensor(ks, dtype=torch.int32, device=a.device)
    d = out if out is not None else torch.empty((len(ks), M, N), dtype=torch.float32, device=a.device)
    _lib.dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, c, d, ks, ks_dev, len(ks), M, N, stream)
    return d


# ---------------------------------------------------------------------------------------------
# The operators around the experts' products
# ---------------------------------------------------------------------------------------------

_TYPES = {torch.bfloat16: 0, torch.float32: 1}       # dg_dtype
_SCORES = {"softmax": 0, "sigmoid": 1}               # dg_score


@functools.lru_cache(maxsize=1024)
def _norm_workspace(T, K):
    return _lib.dg_layer_norm_backward_workspace(T, K)


def _check(name, t, shape=None, dtype=None, device=None):
    """A contiguous CUDA tensor of this shape and dtype (or one of these dtypes) on this device (index)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is wanted")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors are on cuda:{device}")
    if dtype is not None and t.dtype is not dtype and (isinstance(dtype, torch.dtype) or t.dtype not in dtype):
        raise ValueError(f"{name}: dtype {t.dtype}, wanted {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, wanted {shape}")


def _check_2d(name, t, dtype, device=None):
    _check(name, t, None, dtype, device)
    s = t.shape
    if len(s) != 2:
        raise ValueError(f"{name}: two dimensions are wanted, got shape {tuple(s)}")
    _check_sizes(*s)
    return s


def _any_start(entry, *args):
    """entry(*args), and where the C ABI refuses an input that does not start on 16 bytes (a slice of a batch; the refusal
    comes before anything is queued) the same with copies of such inputs. Asking each tensor first costs 0.4 us a call."""
    try:
        entry(*args)
    except _lib.DgError as e:
        if e.status != _lib.DG_ERR_ALIGNMENT:
            raise
        entry(*(a.clone() if isinstance(a, torch.Tensor) and a.data_ptr() % 16 else a for a in args))


def _check_sizes(*sizes):
    """The C ABI takes 32-bit sizes; ctypes would cut larger ones off without a word."""
    if max(sizes) >= 2 ** 31 or min(sizes) < -2 ** 31:
        raise ValueError(f"sizes {sizes} do not fit 32 bits")


def _elsewhere(device, stream):
    """Whether a call has to change the current device or stream first (_on)."""
    return stream is not None or device != torch._C._cuda_getDevice()


def _on(device, stream):
    """Makes the device (an index) and ``stream`` current: kernels run there, and what is allocated inside
    belongs to that stream, so that a workspace is not handed out again while it is in use."""
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{device}")
    return torch.cuda.stream(stream)


# The current stream of a device (index) as a raw handle; through a Stream object it takes 3 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _norm_args(x, weight, bias, rms):
    T, K = _check_2d("x", x, _TYPES)
    if weight is not None:
        _check("weight", weight, (K,), _TYPES, x.get_device())
    if bias is not None:
        if rms:
            raise ValueError("the RMS form takes no bias")
        _check("bias", bias, (K,), weight.dtype if weight is not None else _TYPES, x.get_device())
    w = weight if weight is not None else bias
    return T, K, _TYPES[w.dtype] if w is not None else 0


def layer_norm(x, weight=None, bias=None, eps=1e-5, rms=False, stats=False, out=None, stream=None):
    """Layer norm (or RMS norm) of the rows of x [T,K], bf16 or fp32: y of x's type. weight and bias
    [K] are bf16 or fp32 (both alike). With ``stats`` returns (y, mean, rstd) for layer_norm_backward (mean is
    None in the RMS form). ``out`` may be x."""
    T, K, w_type = _norm_args(x, weight, bias, rms)
    if out is not None:
        _check("out", out, (T, K), x.dtype, x.get_device())
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm(x, weight, bias, eps, rms, stats, out)
    y = out if out is not None else torch.empty_like(x)
    mean = rstd = None
    if stats:
        rstd = x.new_empty(T, dtype=torch.float32)
        mean = None if rms else torch.empty_like(rstd)
    if T:
        _lib.dg_layer_norm(x, weight, bias, y, None, None, mean, rstd, T, K, eps, int(rms), _TYPES[x.dtype], w_type,
                           _raw_stream(dev))
    return (y, mean, rstd) if stats else y


def layer_norm_cast(x, weight=None, bias=None, eps=1e-5, rms=False, stream=None):
    """layer_norm and the per-token FP8 cast of its unrounded result in one pass: (e4m3 [T,K], sfa fp32
    [Kb][pad4(T)], padding zero), the A operand of fp8_gemm_nt. K % 128 == 0."""
    T, K, w_type = _norm_args(x, weight, bias, rms)
    if K % 128:
        raise ValueError(f"K = {K} is not a multiple of 128")
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm_cast(x, weight, bias, eps, rms)
    q = torch.empty_like(x, dtype=torch.uint8)
    sfa = (x.new_zeros if T % 4 else x.new_empty)((K // 128, _pad4(T)), dtype=torch.float32)
    if T:
        _lib.dg_layer_norm(x, weight, bias, None, q, sfa, None, None, T, K, eps, int(rms), _TYPES[x.dtype], w_type,
                           _raw_stream(dev))
    return q, sfa


def layer_norm_backward(dy, x, weight, mean, rstd, bias=True, rms=False, stream=None):
    """Gradients (dx [T,K] of x's type, dw fp32 [K] or None without a weight, db fp32 [K] or None unless
    ``bias``) of layer_norm from dy and the saved mean and rstd (fp32 [T]; mean None in the RMS form)."""
    T, K, w_type = _norm_args(x, weight, None, rms)
    _check("dy", dy, (T, K), x.dtype, x.get_device())
    _check("rstd", rstd, (T,), torch.float32, x.get_device())
    if (mean is None) != bool(rms):
        raise ValueError("mean is wanted unless rms")
    if mean is not None:
        _check("mean", mean, (T,), torch.float32, x.get_device())
    if rms and bias:
        raise ValueError("the RMS form has no bias")
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm_backward(dy, x, weight, mean, rstd, bias, rms)
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight, dtype=torch.float32) if weight is not None else None
    db = x.new_empty(K, dtype=torch.float32) if bias else None
    if T == 0:
        for g in (dw, db):
            if g is not None:
                g.zero_()
        return dx, dw, db
    need = _norm_workspace(T, K) if weight is not None or bias else 0
    ws = x.new_empty(need, dtype=torch.uint8) if need else None
    _lib.dg_layer_norm_backward(dy, x, weight, mean, rstd, dx, dw, db, ws, need, T, K, _TYPES[x.dtype], w_type,
                                _raw_stream(dev))
    return dx, dw, db


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score {score!r}: softmax or sigmoid")
    return _SCORES[score]


def moe_route(logits, k, bias=None, groups=1, topk_groups=1, group_top=1, score="softmax", renorm=True, scale=1.0,
              stream=None):
    """Routing of logits [T,E] (bf16 or fp32) to k experts a token: (weights fp32 [T,k], ids int32 [T,k]).
    The choice goes by score + bias (fp32 [E]) within the topk_groups best groups; the bias is in no
    weight. Places that no expert fills hold id -1 and weight 0."""
    T, E = _check_2d("logits", logits, _TYPES)
    if bias is not None:
        _check("bias", bias, (E,), torch.float32, logits.get_device())
    s = _score(score)
    _check_sizes(k, groups, topk_groups, group_top)
    dev = logits.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return moe_route(logits, k, bias, groups, topk_groups, group_top, score, renorm, scale)
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = torch.empty_like(ids, dtype=torch.float32)
    if T:
        _any_start(_lib.dg_moe_route, logits, bias, ids, weights, T, E, k, groups, topk_groups, group_top, s, int(renorm),
                   scale, _TYPES[logits.dtype], _raw_stream(dev))
    return weights, ids


def moe_route_backward(grad_weights, logits, ids, score="softmax", renorm=True, scale=1.0, stream=None):
    """Gradient of the logits (of their type) from the gradient of moe_route's weights (fp32 [T,k])."""
    T, E = _check_2d("logits", logits, _TYPES)
    _, k = _check_2d("ids", ids, torch.int32, logits.get_device())
    _check("ids", ids, (T, k))
    _check("grad_weights", grad_weights, (T, k), torch.float32, logits.get_device())
    s = _score(score)
    dev = logits.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return moe_route_backward(grad_weights, logits, ids, score, renorm, scale)
    g = torch.empty_like(logits)
    if T:
        _any_start(_lib.dg_moe_route_backward, grad_weights, logits, ids, g, T, E, k, s, int(renorm), scale,
                   _TYPES[logits.dtype], _raw_stream(dev))
    return g


def moe_layout_contiguous(ids, G, M_sum=None, stream=None):
    """Rows of the contiguous layout for expert ids int32 [T,k] (ids outside [0,G) are dropped):
    (dst_rows int32 [T,k], grouped_layout int32 [M_sum], ks int32 [G]). ks are the experts' padded row
    counts. The default M_sum fits any ids."""
    T, k = _check_2d("ids", ids, torch.int32)
    if M_sum is None:
        M_sum = (T * k + 127 * min(G, T * k) + 127) // 128 * 128
    _check_sizes(G, M_sum)
    dev = ids.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return moe_layout_contiguous(ids, G, M_sum)
    dst = torch.empty_like(ids)
    layout = ids.new_empty(M_sum)
    ks = ids.new_empty(G)
    _any_start(_lib.dg_moe_layout_contiguous, ids, dst, layout, ks, T, k, G, M_sum, _raw_stream(dev))
    return dst, layout, ks


def moe_layout_masked(ids, G, M_max, stream=None):
    """Rows of the masked layout for expert ids int32 [T,k] (ids outside [0,G) are dropped):
    (dst_rows int32 [T,k] with row g·M_max + i for expert g's i-th token, masked_m int32 [G])."""
    T, k = _check_2d("ids", ids, torch.int32)
    _check_sizes(G, M_max)
    dev = ids.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return moe_layout_masked(ids, G, M_max)
    dst = torch.empty_like(ids)
    masked_m = ids.new_empty(G)
    _any_start(_lib.dg_moe_layout_masked, ids, dst, masked_m, T, k, G, M_max, _raw_stream(dev))
    return dst, masked_m


def cast_per_token_scatter_topk(x, dst_rows, M, G=1, out=None, stream=None):
    """The per-token FP8 cast of x bf16 [T,K] into each token's rows dst_rows int32 [T,k] of G groups of M
    rows (contiguous: G = 1, M = M_sum; masked: M = M_max): (e4m3 [G·M,K], sfa fp32 [G,Kb,pad4(M)]).
    Rows no token maps to are zero, or keep what ``out`` = (q, sfa) held."""
    T, K = _check_2d("x", x, torch.bfloat16)
    _, k = _check_2d("dst_rows", dst_rows, torch.int32, x.get_device())
    _check("dst_rows", dst_rows, (T, k))
    if K % 128:
        raise ValueError(f"K = {K} is not a multiple of 128")
    _check_sizes(M, G, G * M)
    if out is not None:
        _check("out[0]", out[0], (G * M, K), torch.uint8, x.get_device())
        _check("out[1]", out[1], (G, K // 128, _pad4(M)), torch.float32, x.get_device())
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cast_per_token_scatter_topk(x, dst_rows, M, G, out)
    q, sfa = out if out is not None else (
        x.new_zeros((G * M, K), dtype=torch.uint8),
        torch.zeros((G, K // 128, _pad4(M)), dtype=torch.float32, device=x.device))
    if T and k and G * M:
        _lib.dg_cast_fp8_per_token_scatter_topk(x, dst_rows, q, sfa, T, k, G, M, K, _raw_stream(dev))
    return q, sfa


def _combine_sizes(d, dst_rows):
    _check("d", d, None, torch.bfloat16)
    if d.dim() < 2:
        raise ValueError(f"d: two dimensions or more are wanted, got shape {tuple(d.shape)}")
    T, k = _check_2d("dst_rows", dst_rows, torch.int32, d.get_device())
    N = d.shape[-1]
    R = d.numel() // max(N, 1)
    _check_sizes(N, R)
    return T, k, N, R


def moe_combine(d, dst_rows, weights=None, c=None, out=None, stream=None):
    """y[t] = c[t] + sum_j weights[t,j]·d[dst_rows[t,j]] (bf16 [T,N]; d bf16 with rows of N, of any leading
    shape; negative rows are left out). ``out`` may be c. Without weights (ones) this is also the
    gradient of the dispatch."""
    T, k, N, R = _combine_sizes(d, dst_rows)
    if weights is not None:
        _check("weights", weights, (T, k), torch.float32, d.get_device())
    if c is not None:
        _check("c", c, (T, N), torch.bfloat16, d.get_device())
    if out is not None:
        _check("out", out, (T, N), torch.bfloat16, d.get_device())
    dev = d.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return moe_combine(d, dst_rows, weights, c, out)
    y = out if out is not None else d.new_empty((T, N)) if c is None else torch.empty_like(c)
    if T:
        _lib.dg_moe_combine(d, dst_rows, weights, c, y, T, k, N, R, _raw_stream(dev))
    return y


def moe_combine_backward(grad_y, d, dst_rows, weights=None, grouped_layout=None, stream=None):
    """Gradients (grad_d like d, grad_weights fp32 [T,k]) of moe_combine. Rows of grad_d that no pair
    maps to: with grouped_layout (int32 [M_sum]) its negative rows are zero and every other row has a
    pair; without it all of them are zero."""
    T, k, N, R = _combine_sizes(d, dst_rows)
    _check("grad_y", grad_y, (T, N), torch.bfloat16, d.get_device())
    if weights is not None:
        _check("weights", weights, (T, k), torch.float32, d.get_device())
    if grouped_layout is not None:
        _check("grouped_layout", grouped_layout, (R,), torch.int32, d.get_device())
    dev = d.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return moe_combine_backward(grad_y, d, dst_rows, weights, grouped_layout)
    gd = (torch.zeros_like if grouped_layout is None else torch.empty_like)(d)
    gw = torch.empty_like(dst_rows, dtype=torch.float32)
    if T or (R and grouped_layout is not None):
        _lib.dg_moe_combine_backward(grad_y, d, dst_rows, weights, grouped_layout, gd, gw, T, k, N, R, _raw_stream(dev))
    return gd, gw
