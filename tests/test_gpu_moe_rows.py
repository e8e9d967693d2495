"""Rows of the grouped layouts, the top-k dispatch cast and the weighted combine with its gradient, each
against a plain implementation; then all of them together around the framework's grouped GEMMs."""
import threading

import numpy as np
import pytest
import torch

from moe_grouped_gemm_sm_b200 import _lib, build, ops, synth
from tests.gpu_util import assert_close, bf16_dev, bf16_host_f64, dev, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def place(ids, G, M, masked):
    """(dst, grouped_layout or None, counts, lost) by walking the pairs in order."""
    flat = ids.reshape(-1)
    count = np.zeros(G, np.int64)
    for e in flat:
        if 0 <= e < G:
            count[e] += 1
    padded = (count + 127) // 128 * 128
    first = np.arange(G) * M if masked else np.concatenate([[0], np.cumsum(padded)[:-1]])
    nxt, dst, lost = first.copy(), np.full(flat.size, -1, np.int64), False
    for i, e in enumerate(flat):
        if 0 <= e < G:
            if nxt[e] < (first[e] + M if masked else M):
                dst[i] = nxt[e]
            else:
                lost = True
            nxt[e] += 1
    if masked:
        return dst.reshape(ids.shape), None, np.minimum(count, M), lost
    layout = np.full(M, -1, np.int64)
    for g in range(G):
        layout[first[g]:min(M, first[g] + count[g])] = g
    return dst.reshape(ids.shape), layout, np.clip(np.minimum(padded, M - first), 0, None), lost


def expert_ids(T, k, G, seed=0, wild=False):
    rng = np.random.default_rng(seed * 1000 + T + k + G)
    p = rng.exponential(size=G) + 0.01
    ids = rng.choice(G, size=(T, k), p=p / p.sum()).astype(np.int32)     # an expert may come twice in a token
    if wild and T:
        ids[rng.random((T, k)) < 0.2] = -1
        ids[rng.random((T, k)) < 0.05] = G
        ids[0, 0], ids[-1, -1] = 2 ** 31 - 1, -2 ** 31
    return ids


LAYOUTS = [(0, 1, 1), (1, 1, 1), (1, 8, 256), (5, 2, 3), (129, 1, 1), (128, 8, 16), (256, 8, 33), (255, 8, 64), (257, 8, 64),
           (2049, 1, 1), (700, 6, 1024), (5000, 8, 256), (33333, 3, 7), (40000, 7, 300)]


@pytest.mark.parametrize("T,k,G", LAYOUTS)
@pytest.mark.parametrize("wild", [False, True])
def test_contiguous_layout(T, k, G, wild):
    ids = expert_ids(T, k, G, wild=wild)
    dst, layout, ks = ops.moe_layout_contiguous(dev(ids), G)
    rd, rl, rk, lost = place(ids, G, layout.numel(), False)
    assert not lost
    assert np.array_equal(host(dst), rd) and np.array_equal(host(layout), rl) and np.array_equal(host(ks), rk)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("T,k,G", LAYOUTS)
@pytest.mark.parametrize("wild", [False, True])
def test_masked_layout(T, k, G, wild):
    ids = expert_ids(T, k, G, seed=1, wild=wild)
    M = max(1, T * k)
    dst, mm = ops.moe_layout_masked(dev(ids), G, M)
    rd, _, rm, lost = place(ids, G, M, True)
    assert not lost and np.array_equal(host(dst), rd) and np.array_equal(host(mm), rm)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("T,k,G", [(300, 4, 9), (5000, 8, 20)])
def test_layouts_that_are_too_small(T, k, G):
    ids = expert_ids(T, k, G, seed=2)
    for M in (0, 128, 1024):
        dst, layout, ks = ops.moe_layout_contiguous(dev(ids), G, M_sum=M)
        rd, rl, rk, lost = place(ids, G, M, False)
        assert lost and _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
        assert np.array_equal(host(dst), rd) and np.array_equal(host(layout), rl) and np.array_equal(host(ks), rk)
    for M in (0, 1, 50):
        dst, mm = ops.moe_layout_masked(dev(ids), G, M)
        rd, _, rm, lost = place(ids, G, M, True)
        assert lost and _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
        assert np.array_equal(host(dst), rd) and np.array_equal(host(mm), rm)


@pytest.mark.parametrize("T,k,G,M,K", [(1, 1, 1, 128, 128), (7, 8, 1, 1024, 384), (200, 3, 1, 1152, 7168), (64, 8, 16, 50, 640),
                                       (33, 2, 5, 33, 256), (1500, 4, 1, 6272, 1024), (1, 32, 2, 32, 2048), (2, 100, 1, 512, 256),
                                       (3, 7, 4, 9, 17024), (400, 8, 1, 3584, 2048)])
def test_dispatch_cast(oracle, T, k, G, M, K):
    """Bit for bit the per-token cast in the rows of the pairs; every other row as it was."""
    x = synth.normal_bf16(T + K, (T, K))
    x[0, :128] = 0
    rng = np.random.default_rng(T)
    dst = rng.permutation(G * M)[:T * k].astype(np.int32).reshape(T, k)
    dst[rng.random((T, k)) < 0.1] = -1
    q = torch.full((G * M, K), 77, dtype=torch.uint8, device="cuda")
    sfa = torch.full((G, K // 128, (M + 3) // 4 * 4), -5.0, device="cuda")
    got = ops.cast_per_token_scatter_topk(bf16_dev(x), dev(dst), M, G=G, out=(q, sfa))
    assert got[0] is q and got[1] is sfa
    qo, so = oracle.cast_per_token(x)
    rq, rs = np.full((G * M, K), 77, np.uint8), np.full(tuple(sfa.shape), -5.0, np.float32)
    for t in range(T):
        for r in dst[t]:
            if r >= 0:
                rq[r] = qo[t]
                rs[r // M, :, r % M] = so[:, t]
    assert np.array_equal(host(q), rq) and np.array_equal(host(sfa), rs)
    assert _lib.dg_get_device_error() == _lib.DG_OK
    q2, sfa2 = ops.cast_per_token_scatter_topk(bf16_dev(x), dev(dst), M, G=G)
    assert np.array_equal(host(q2), np.where((rq == 77).all(1, keepdims=True), 0, rq))
    assert np.array_equal(host(sfa2), np.where(rs == -5, 0, rs))


def test_dispatch_cast_leaves_out_rows_outside():
    x = synth.normal_bf16(3, (4, 256))
    dst = np.array([[0, 8], [2 ** 31 - 1, 1], [-7, 2], [3, 100]], np.int32)
    q, sfa = ops.cast_per_token_scatter_topk(bf16_dev(x), dev(dst), 4, G=2)
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
    inside = np.where((dst < 0) | (dst >= 8), -1, dst).astype(np.int32)
    q2, sfa2 = ops.cast_per_token_scatter_topk(bf16_dev(x), dev(inside), 4, G=2)
    assert torch.equal(q, q2) and torch.equal(sfa, sfa2) and _lib.dg_get_device_error() == _lib.DG_OK


def test_dispatch_cast_behind_2_to_31_codes():
    """Code offsets that pass 32 bits: the last rows of 300000 rows of 8192 codes."""
    R, K = 300000, 8192
    x = synth.normal_bf16(11, (3, K))
    dst = np.array([[R - 1], [262144], [0]], np.int32)
    q = torch.zeros((R, K), dtype=torch.uint8, device="cuda")
    sfa = torch.zeros((1, K // 128, R), device="cuda")
    ops.cast_per_token_scatter_topk(bf16_dev(x), dev(dst), R, out=(q, sfa))
    ref, _ = ops.cast_per_token(bf16_dev(x))
    rows = torch.from_numpy(dst[:, 0]).long().cuda()
    assert torch.equal(q[rows], ref) and int(q.count_nonzero()) == int(ref.count_nonzero())
    d = q.view(torch.bfloat16)                    # the same rows as bf16 [R, K/2], 2.5 GB
    y = ops.moe_combine(d, dev(dst))
    nan = torch.isnan(d[rows])
    assert torch.equal(torch.where(nan, 0, y), torch.where(nan, 0, d[rows]))


COMBINE = [(1, 1, 8, 1), (1, 8, 7168, 8), (5, 3, 264, 20), (64, 8, 7168, 600), (37, 32, 1024, 1300), (300, 2, 72, 700),
           (700, 6, 2048, 4300), (2, 5, 20000, 10)]


def pairs(T, k, R, seed=0):
    rng = np.random.default_rng(seed + T + R)
    dst = rng.permutation(max(R, T * k))[:T * k].reshape(T, k)
    dst[dst >= R] = -1
    if T > 2:
        dst[rng.random((T, k)) < 0.1] = -1
        dst[1] = -1                               # a token without any row
    return dst.astype(np.int32)


def combine_inputs(T, k, N, R, seed=0):
    g = torch.Generator().manual_seed(seed + T + N)
    d = torch.randn(R, N, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g)
    c = torch.randn(T, N, generator=g).bfloat16()
    return d, torch.from_numpy(pairs(T, k, R, seed)), w, c


@pytest.mark.parametrize("T,k,N,R", COMBINE)
def test_combine(T, k, N, R):
    d, dst, w, c = combine_inputs(T, k, N, R)
    unread = torch.ones(R, dtype=torch.bool)
    unread[dst[dst >= 0].long()] = False
    d[unread] = float("nan")                      # rows that no pair names are not read
    rows = torch.where((dst >= 0).unsqueeze(2), d.double()[dst.clamp(min=0).long()], 0)
    for wt, cc in ((w, c), (w, None), (None, c), (None, None)):
        y = ops.moe_combine(d.cuda(), dst.cuda(), None if wt is None else wt.cuda(), c=None if cc is None else cc.cuda())
        terms = rows * (1 if wt is None else wt.double().unsqueeze(2))
        ref = terms.sum(1) + (0 if cc is None else cc.double())
        # k + 1 fp32 additions and products, then half a bf16 step
        tol = (k + 2) * U * (terms.abs().sum(1) + (0 if cc is None else cc.double().abs()))
        assert ((y.cpu().double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all()
    cd = c.cuda()
    y = ops.moe_combine(d.cuda(), dst.cuda(), w.cuda(), c=cd)
    assert ops.moe_combine(d.cuda(), dst.cuda(), w.cuda(), c=cd, out=cd) is cd and torch.equal(cd, y)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("T,k,N,R", COMBINE)
def test_combine_backward(T, k, N, R):
    d, dst, w, _ = combine_inputs(T, k, N, R, seed=1)
    gy = torch.randn(T, N, generator=torch.Generator().manual_seed(2)).bfloat16()
    on = dst >= 0
    layout = torch.full((R,), -1, dtype=torch.int32)
    layout[dst[on].long()] = 3
    for wt in (w, None):
        wd = torch.ones(T, k, dtype=torch.float64) if wt is None else wt.double()
        terms = wd.unsqueeze(2) * gy.double().unsqueeze(1)
        rgd = torch.zeros(R, N, dtype=torch.float64)
        rgd[dst[on].long()] = terms[on]
        prod = d.double()[dst.clamp(min=0).long()] * gy.double().unsqueeze(1)
        rgw = prod.sum(2) * on
        for lay in (layout, None):
            gd, gw = ops.moe_combine_backward(gy.cuda(), d.cuda(), dst.cuda(), None if wt is None else wt.cuda(),
                                              grouped_layout=None if lay is None else lay.cuda())
            assert ((gd.cpu().double() - rgd).abs() <= (2.0 ** -8 + 2 * U) * rgd.abs()).all()
            # a dot product of N terms: at most N - 1 additions, one rounding a term
            assert ((gw.cpu().double() - rgw).abs() <= N * U * prod.abs().sum(2)).all()
            assert not gw.cpu()[~on].any()
    assert _lib.dg_get_device_error() == _lib.DG_OK


def test_combine_gradients_against_differences():
    """y is linear in d and in the weights, so a difference of any step is the derivative: the step itself
    is the perturbation. Kernels' roundings: half a bf16 step of each grad_d, N·u of each dot product."""
    T, k, N, R = 9, 3, 64, 40
    d, dst, w, _ = combine_inputs(T, k, N, R, seed=5)
    gen = torch.Generator().manual_seed(7)
    gy, vd, vw = torch.randn(T, N, generator=gen).bfloat16(), torch.randn(R, N, generator=gen), torch.randn(T, k, generator=gen)
    gd, gw = ops.moe_combine_backward(gy.cuda(), d.cuda(), dst.cuda(), w.cuda())
    on = (dst >= 0).unsqueeze(2)

    def f(dd, ww):
        return float(((torch.where(on, dd[dst.clamp(min=0).long()], 0) * ww.unsqueeze(2)).sum(1) * gy.double()).sum())
    dd, ww = d.double(), w.double()
    num_d = f(dd + vd.double(), ww) - f(dd, ww)
    num_w = f(dd, ww + vw.double()) - f(dd, ww)
    gd, gw = gd.cpu().double(), gw.cpu().double()
    assert abs(float((gd * vd).sum()) - num_d) <= float((gd.abs() * vd.abs()).sum()) * 2.0 ** -8 * 1.01 + 1e-9
    size = (torch.where(on, dd[dst.clamp(min=0).long()], 0) * gy.double().unsqueeze(1)).abs().sum(2)
    assert abs(float((gw * vw).sum()) - num_w) <= float((size * vw.abs()).sum()) * N * U + 1e-9


def test_combine_leaves_out_rows_outside():
    d, dst, w, c = combine_inputs(4, 2, 64, 8)
    dst = torch.tensor([[0, 8], [2 ** 31 - 1, 1], [-7, 2], [3, 4]], dtype=torch.int32)
    inside = torch.where((dst < 0) | (dst >= 8), torch.tensor(-1, dtype=torch.int32), dst)
    args = (d.cuda(), dst.cuda(), w.cuda())
    y = ops.moe_combine(*args)
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
    assert torch.equal(y, ops.moe_combine(d.cuda(), inside.cuda(), w.cuda()))
    got = ops.moe_combine_backward(c.cuda(), *args)
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
    ref = ops.moe_combine_backward(c.cuda(), d.cuda(), inside.cuda(), w.cuda())
    assert all(torch.equal(p, q) for p, q in zip(got, ref)) and _lib.dg_get_device_error() == _lib.DG_OK


def test_no_tokens():
    d = torch.ones(256, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    layout = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    assert ops.moe_combine(d, none).shape == (0, 64)
    gd, gw = ops.moe_combine_backward(e, d, none, grouped_layout=layout)
    assert not gd.any() and gw.shape == (0, 4)
    y = ops.moe_combine(d[:0], torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), c=d[:3].contiguous())
    assert torch.equal(y, d[:3])
    q, sfa = ops.cast_per_token_scatter_topk(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), none, 128)
    assert not q.any()


def moe_forward(h, logits, bias, w1, s1, w2, s2, k, G, c, masked):
    """One MoE layer out of the framework's calls (two products an expert), contiguous or masked."""
    wt, ids = ops.moe_route(logits, k, bias=bias, groups=4, topk_groups=2, group_top=2, score="sigmoid")
    T = h.shape[0]
    if masked:
        dst, mm = ops.moe_layout_masked(ids, G, T)
        q, sfa = ops.cast_per_token_scatter_topk(h, dst, T, G=G)
        a = ops.m_grouped_fp8_gemm_nt_masked(q.view(G, T, -1), sfa, w1, s1, mm, T)
        q, sfa = ops.cast_per_token(a)
        d = ops.m_grouped_fp8_gemm_nt_masked(q, sfa, w2, s2, mm, T)
        return ops.moe_combine(d, dst, wt, c=c), dst, wt
    dst, layout, ks = ops.moe_layout_contiguous(ids, G)
    q, sfa = ops.cast_per_token_scatter_topk(h, dst, layout.numel())
    a = ops.m_grouped_fp8_gemm_nt_contiguous(q, sfa[0], w1, s1, layout)
    q, sfa = ops.cast_per_token(a)
    d = ops.m_grouped_fp8_gemm_nt_contiguous(q, sfa, w2, s2, layout)
    return ops.moe_combine(d, dst, wt, c=c), dst, wt, layout, ks, d


def test_a_layer_together(oracle):
    """norm -> route -> layout -> dispatch -> two grouped products -> combine, contiguous and masked; each
    expert's products recomputed by the oracle from the codes that the casts give for the same rows."""
    T, K, I, G, k = 150, 512, 256, 16, 4
    g = torch.Generator().manual_seed(21)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    nw = (1 + 0.1 * torch.randn(K, generator=g)).cuda()
    logits = torch.randn(T, G, generator=g).cuda()
    bias = (0.05 * torch.randn(G, generator=g)).cuda()
    b1, b2 = synth.normal_bf16(31, (G, I, K), sigma=K ** -0.5), synth.normal_bf16(32, (G, K, I), sigma=I ** -0.5)
    w1, s1 = ops.cast_per_block(bf16_dev(b1))
    w2, s2 = ops.cast_per_block(bf16_dev(b2))
    h = ops.layer_norm(x, nw, rms=True)
    y, dst, wt, layout, ks, _ = moe_forward(h, logits, bias, w1, s1, w2, s2, k, G, x, False)
    ym, dstm, wtm = moe_forward(h, logits, bias, w1, s1, w2, s2, k, G, x, True)
    torch.cuda.synchronize()
    assert _lib.dg_get_device_error() == _lib.DG_OK
    _, ids = ops.moe_route(logits, k, bias=bias, groups=4, topk_groups=2, group_top=2, score="sigmoid")
    ids, hb = host(ids), host(h.view(torch.int16)).view(np.uint16)
    qh, sh = oracle.cast_per_token(hb)
    w1h, s1h, w2h, s2h = host(w1), host(s1), host(w2), host(s2)
    ref, size = bf16_host_f64(x), np.abs(bf16_host_f64(x))
    for e in range(G):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        m4 = (t.size + 3) // 4 * 4
        sf = np.zeros((K // 128, m4), np.float32)
        sf[:, :t.size] = sh[:, t]
        a = oracle.gemm_nt(np.ascontiguousarray(qh[t]), sf, w1h[e], s1h[e], None)
        # the second product's codes are those of the bf16 result, at most a bf16 step from this one's
        q2, sf2 = oracle.cast_per_token(synth.f32_to_bf16_bits(a.astype(np.float32)))
        d = oracle.gemm_nt(q2, sf2, w2h[e], s2h[e], None)
        wj = host(wt)[t, j].astype(np.float64)[:, None]
        np.add.at(ref, t, wj * d)
        np.add.at(size, t, wj * np.sqrt(np.mean(d ** 2)))
    for got in (bf16_host_f64(y), bf16_host_f64(ym)):
        # a code of the second product may fall to the next one (2^-3 of a few values, averaged over I of
        # them), and y is rounded to bf16: 2^-8 of it, and 2^-4 of the products' size as a whole
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -4 * size).all()
        assert np.sqrt(np.mean((got - ref) ** 2)) <= 2.0 ** -8 * np.sqrt(np.mean(ref ** 2)) + 2.0 ** -7 * np.sqrt(np.mean(size ** 2))
    # the two layouts hold the same rows, so the same codes and products
    assert torch.equal(wt, wtm)
    assert ((y.double() - ym.double()).abs() <= 2.0 ** -7 * y.double().abs() + 2.0 ** -4 * torch.from_numpy(size).cuda()).all()


def test_a_backward_pass_together():
    """combine's gradient feeds the K-grouped weight gradient: rows of padding are zero there, ks are the
    layout's, and the dispatch's gradient is a combine without weights."""
    T, N, K, G, k = 200, 128, 256, 6, 2
    gen = torch.Generator().manual_seed(8)
    ids = torch.from_numpy(expert_ids(T, k, G, seed=5)).cuda()
    x = torch.randn(T, K, generator=gen).bfloat16().cuda()
    dst, layout, ks = ops.moe_layout_contiguous(ids, G)
    R = layout.numel()
    d = torch.randn(R, N, generator=gen).bfloat16().cuda()
    wt = torch.rand(T, k, generator=gen).cuda()
    gy = torch.randn(T, N, generator=gen).bfloat16().cuda()
    gd, gw = ops.moe_combine_backward(gy, d, dst, wt, grouped_layout=layout)
    assert not gd[layout < 0].any()
    # the experts' inputs in bf16 (zero in the padding): the weight gradient's other operand
    xr = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    xr[dst.long().reshape(-1)] = x.repeat_interleave(k, 0)
    used = int(ks.sum())
    a, sfa = ops.cast_per_channel(gd[:used].contiguous())
    b, sfb = ops.cast_per_channel(xr[:used].contiguous())
    dw = ops.k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, ks.tolist())
    ref = torch.zeros(G, N, K, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref)
    for e in range(G):
        t, j = (ids == e).nonzero(as_tuple=True)
        ge, xe = wt[t, j].double()[:, None] * gy[t].double(), x[t].double()
        ref[e], size[e] = ge.t() @ xe, ge.abs().t() @ xe.abs()
    # two operands, each within an e4m3 half step (2^-4) of itself and 2^-10·(amax/448) near zero
    assert ((dw.double() - ref).abs() <= (2 * 2.0 ** -4 + 2.0 ** -7) * size + 0.02).all()
    gx = ops.moe_combine(xr, dst)                 # the dispatch's gradient: the sum of the k rows
    assert ((gx.double() - k * x.double()).abs() <= 2.0 ** -8 * (k * x.double()).abs()).all()


def test_streams_and_graphs():
    T, K, I, G, k = 96, 256, 128, 8, 4
    gen = torch.Generator().manual_seed(9)
    h = torch.randn(T, K, generator=gen).bfloat16().cuda()
    logits, bias = torch.randn(T, G, generator=gen).cuda(), torch.zeros(G).cuda()
    w1, s1 = ops.cast_per_block(torch.randn(G, I, K, generator=gen).bfloat16().cuda())
    w2, s2 = ops.cast_per_block(torch.randn(G, K, I, generator=gen).bfloat16().cuda())
    big = torch.from_numpy(expert_ids(4000, 4, G)).cuda()   # layouts with a workspace

    def step():
        y, dst, wt, layout, ks, d = moe_forward(h, logits, bias, w1, s1, w2, s2, k, G, h, False)
        gd, gw = ops.moe_combine_backward(h, d, dst, wt, grouped_layout=layout)
        return (y, dst, wt, layout, ks, gw, gd * (layout[:, None] >= 0),
                *ops.moe_layout_contiguous(big, G), *ops.moe_layout_masked(big, G, 16000))
    ref = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    q, sfa = ops.cast_per_token_scatter_topk(h, ref[1], ref[3].numel())
    d = torch.randn(ref[3].numel(), K, generator=gen).bfloat16().cuda()
    plain = [*ops.moe_layout_contiguous(big, G), *ops.moe_layout_masked(big, G, 16000), q, sfa,
             ops.moe_combine(d, ref[1], ref[2]), *ops.moe_combine_backward(h, d, ref[1], ref[2])]
    torch.cuda.synchronize()
    for st in (s, s.cuda_stream, 0):                        # the stream as an argument
        got = [*ops.moe_layout_contiguous(big, G, stream=st), *ops.moe_layout_masked(big, G, 16000, stream=st),
               *ops.cast_per_token_scatter_topk(h, ref[1], ref[3].numel(), stream=st),
               ops.moe_combine(d, ref[1], ref[2], stream=st), *ops.moe_combine_backward(h, d, ref[1], ref[2], stream=st)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, plain))
    pool, graphs = None, []
    for _ in range(2):                                      # two graphs on one memory pool: their workspaces may be the same
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = step()
        pool = graph.pool()
        graphs.append((graph, out))
    for graph, out in graphs + graphs:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, ref))
    assert _lib.dg_get_device_error() == _lib.DG_OK


def test_two_threads_at_once():
    """Calls from two host threads, each on a stream of its own, give what one thread's calls give."""
    T, K, G, k = 300, 512, 32, 4
    gen = torch.Generator().manual_seed(12)
    data = [(torch.randn(T, K, generator=gen).bfloat16().cuda(), torch.randn(T, G, generator=gen).cuda()) for _ in range(2)]

    def step(x, logits):
        h, mean, rstd = ops.layer_norm(x, stats=True)
        wt, ids = ops.moe_route(logits, k, score="sigmoid")
        dst, layout, ks = ops.moe_layout_contiguous(ids, G)
        q, sfa = ops.cast_per_token_scatter_topk(h, dst, layout.numel())
        d = torch.zeros(layout.numel(), K, dtype=torch.bfloat16, device="cuda")
        d[dst.long().reshape(-1)] = h.repeat_interleave(k, 0)
        y = ops.moe_combine(d, dst, wt, c=x)
        gd, gw = ops.moe_combine_backward(x, d, dst, wt, grouped_layout=layout)
        gl = ops.moe_route_backward(gw, logits, ids, score="sigmoid")
        dx, _, db = ops.layer_norm_backward(y, x, None, mean, rstd)
        return h, wt, ids, dst, layout, ks, q, sfa, y, gw, gl, dx, db
    refs = [step(*v) for v in data]
    torch.cuda.synchronize()
    streams, bad = [torch.cuda.Stream() for _ in data], []

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                out = step(*data[i])
                streams[i].synchronize()
                if not all(torch.equal(p, q) for p, q in zip(out, refs[i])):
                    bad.append(i)
                streams[i].synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and _lib.dg_get_device_error() == _lib.DG_OK


def test_refusals():
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for call in (lambda: ops.moe_layout_contiguous(ids.long(), 4), lambda: ops.moe_layout_contiguous(ids[0], 4),
                 lambda: ops.moe_layout_masked(ids.t(), 4, 8), lambda: ops.cast_per_token_scatter_topk(x.float(), ids, 128),
                 lambda: ops.cast_per_token_scatter_topk(x[:, :100].contiguous(), ids, 128),
                 lambda: ops.cast_per_token_scatter_topk(x, ids[:2], 128),
                 lambda: ops.cast_per_token_scatter_topk(x, ids, 128, out=(x, x)), lambda: ops.moe_combine(x.float(), ids),
                 lambda: ops.moe_combine(x, ids.long()), lambda: ops.moe_combine(x, ids, w[:2]),
                 lambda: ops.moe_combine(x, ids, c=x[:2]), lambda: ops.moe_combine(x, ids, out=x[:2]),
                 lambda: ops.moe_combine_backward(x[:2], x, ids), lambda: ops.moe_combine_backward(x, x, ids, w.double()),
                 lambda: ops.moe_combine_backward(x, x, ids, grouped_layout=ids[:, 0].contiguous()[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.moe_layout_contiguous(ids, 0), lambda: ops.moe_layout_contiguous(ids, 2000),
                 lambda: ops.moe_layout_contiguous(ids, 4, M_sum=100), lambda: ops.moe_layout_masked(ids, 4, -1),
                 lambda: ops.moe_combine(x[:, :12].contiguous(), ids), lambda: ops.moe_combine(x, ids[:, :0].contiguous())):
        with pytest.raises((_lib.DgError, RuntimeError)):
            call()


def test_masked_rows_next_to_2_to_31():
    """The last expert of 1024 with more pairs than M_max = 2^21 - 1: the pairs beyond it get -1, although the rows they
    would have pass 2^31."""
    G, M, n = 1024, 2 ** 21 - 1, 2 ** 21 + 5000
    ids = torch.full((n // 8, 8), G - 1, dtype=torch.int32, device="cuda")
    ids[0] = 0
    dst, mm = ops.moe_layout_masked(ids, G, M)
    place = torch.arange(n - 8, device="cuda")
    ref = torch.cat([torch.arange(8, device="cuda"), torch.where(place < M, (G - 1) * M + place, -1)])
    assert torch.equal(dst.reshape(-1).long(), ref)
    assert mm.tolist() == [8] + [0] * (G - 2) + [M]
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE


def shifted(t, by=1):
    """The same values in memory that does not start on a 16-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    s = buf[by:].view(t.shape)
    s.copy_(t)
    assert s.data_ptr() % 16 and s.is_contiguous()
    return s


@pytest.mark.parametrize("stream", [False, True])
def test_slices_of_a_batch(stream):
    """ids, logits, biases and gradients of the routing and the layouts may start anywhere in a tensor: a slice of a batch
    gives what a copy of it gives."""
    T, E, k = 37, 48, 3
    g = torch.Generator().manual_seed(13)
    gw, bias = torch.randn(T, k, generator=g).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()
    st = torch.cuda.Stream() if stream else None
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(T, E, generator=g).to(dtype).cuda()
        w, ids = ops.moe_route(x, k, bias=bias, groups=6, topk_groups=3)
        ref = [w, ids, ops.moe_route_backward(gw, x, ids), *ops.moe_layout_contiguous(ids, E), *ops.moe_layout_masked(ids, E, T)]
        torch.cuda.synchronize()
        xs, bs, gs, si = shifted(x), shifted(bias), shifted(gw), shifted(ids)
        torch.cuda.synchronize()
        got = [*ops.moe_route(xs, k, bias=bs, groups=6, topk_groups=3, stream=st), ops.moe_route_backward(gs, xs, si, stream=st),
               *ops.moe_layout_contiguous(si, E, stream=st), *ops.moe_layout_masked(si, E, T, stream=st)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
        assert torch.equal(ops.moe_route_backward(gw, x, si), ref[2])
    assert torch.equal(ops.moe_layout_masked(ids[1:], E, T)[1], ops.moe_layout_masked(ids[1:].clone(), E, T)[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*ops.moe_layout_contiguous(si, E), ops.moe_route_backward(gs, xs, si)]
    si.fill_(-1)
    si.copy_(ids)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, [*ref[3:6], ref[2]]))
    assert _lib.dg_get_device_error() == _lib.DG_OK
