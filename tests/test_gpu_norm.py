"""Layer norm and RMS norm (forward, FP8 cast epilogue, backward) against their formulas in 64 bits.

Tolerances count roundings. u = 2^-24 is half a step of fp32. A sum of K terms is taken as at
most 32 (a thread) + 5 (its warp) + 32 (the warps) additions one after another, so a mean is
within 72u of the mean of the magnitudes; every other step adds a few u. With 80u for all of
them: |dy| <= 80u·(|xh·w| + r·|w|·mean|x| + |b|), and half a step of the output type on top."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_sm_b200 import _lib, build, ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def make(T, K, xt, wt, rms, seed=0, weight=True, bias=True):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + K)
    x = (torch.randn(T, K, generator=g) * (0.3 + torch.rand(T, 1, generator=g) * 3) + 0.4).to(xt)
    if K > 5:
        x[:, 5] *= 20
    w = (1 + 0.3 * torch.randn(K, generator=g)).to(wt) if weight else None
    b = (0.5 * torch.randn(K, generator=g)).to(wt) if bias and not rms else None
    return x, w, b


def ref_forward(x, w, b, eps, rms):
    x = x.double()
    mu = torch.zeros(x.shape[0], 1, dtype=torch.float64) if rms else x.mean(1, keepdim=True)
    r = 1 / ((x - mu).square().mean(1, keepdim=True) + eps).sqrt()
    xh = (x - mu) * r
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else b.double()
    tol = 80 * U * ((xh * w).abs() + r * w.abs() * x.abs().mean(1, keepdim=True) + b.abs())
    return xh * w + b, mu[:, 0], r[:, 0], tol


def cuda(t):
    return None if t is None else t.cuda()


SHAPES = [(1, 1), (3, 2), (2, 7), (9, 64), (5, 129), (17, 1000), (300, 1001), (777, 1001), (1, 7168), (33, 2048), (311, 7168),
          (7, 4097), (2, 8191), (600, 24), (1000, 128), (333, 256), (700, 512), (3, 16384), (310, 16384), (301, 12296), (2, 20001), (2, 32768), (300, 32768), (299, 260), (3, 9001), (300, 9001), (2, 8540), (297, 20000)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [False, True])
def test_forward(T, K, xt, rms):
    for wt, weight, bias in ((torch.float32, True, True), (torch.bfloat16, True, False), (torch.bfloat16, False, True)):
        x, w, b = make(T, K, xt, wt, rms, weight=weight, bias=bias)
        y, mean, rstd = ops.layer_norm(cuda(x), cuda(w), cuda(b), eps=1e-5, rms=rms, stats=True)
        ref, mu, r, tol = ref_forward(x, w, b, 1e-5, rms)
        assert y.dtype == xt and ((y.cpu().double() - ref).abs() <= tol + STEP[xt] * (ref.abs() + tol)).all()
        # r: the mean square within 80u and twice the mean's error over the deviation
        mabs = x.double().abs().mean(1)
        assert ((rstd.cpu().double() - r).abs() <= 80 * U * r * (1 + r * mabs)).all()
        if rms:
            assert mean is None
        else:
            assert ((mean.cpu().double() - mu).abs() <= 80 * U * mabs).all()


def test_forward_in_place_and_no_rows():
    x, w, b = make(70, 520, torch.bfloat16, torch.float32, False)
    ref = ops.layer_norm(cuda(x), cuda(w), cuda(b))
    xd = cuda(x)
    assert ops.layer_norm(xd, cuda(w), cuda(b), out=xd) is xd and torch.equal(xd, ref)
    for T, K, rms in ((400, 1024, False), (401, 777, False), (350, 128, True), (300, 8200, True)):   # many rows
        x, w, b = make(T, K, torch.bfloat16, torch.float32, rms, seed=8)
        ref = ops.layer_norm(cuda(x), cuda(w), cuda(b), rms=rms)
        xd = cuda(x)
        assert ops.layer_norm(xd, cuda(w), cuda(b), rms=rms, out=xd) is xd and torch.equal(xd, ref)
    e = torch.empty(0, 64, device="cuda")
    assert ops.layer_norm(e).shape == (0, 64)
    dx, dw, db = ops.layer_norm_backward(e, e, torch.ones(64, device="cuda"), e[:, 0], e[:, 0])
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_constant_rows_and_large_offsets():
    """A constant row has deviation 0 (r = 1/sqrt(eps)); a large mean must not eat the deviation."""
    x = torch.full((4, 768), 3.0)
    x[1] = 0
    x[2] = 1000 + torch.linspace(-1, 1, 768)
    x[3] = -5e4
    y = ops.layer_norm(x.cuda(), eps=1e-5).cpu().double()
    ref, _, _, tol = ref_forward(x, None, None, 1e-5, False)
    assert ((y - ref).abs() <= tol + U).all()
    y = ops.layer_norm(x.cuda(), eps=1e-5, rms=True).cpu().double()
    ref, _, _, tol = ref_forward(x, None, None, 1e-5, True)
    assert ((y - ref).abs() <= tol + U).all()


@pytest.mark.parametrize("T,K", [(1, 128), (5, 256), (6, 1024), (16, 7168), (301, 7168), (1000, 128), (3, 20480), (303, 1152), (401, 256),
                                 (310, 512), (300, 640), (300, 16384), (297, 8320)])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [False, True])
def test_cast(T, K, xt, rms):
    x, w, b = make(T, K, xt, torch.bfloat16, rms, seed=2)
    q, sfa = ops.layer_norm_cast(cuda(x), cuda(w), cuda(b), rms=rms)
    ref, _, _, tol = ref_forward(x, w, b, 1e-5, rms)
    code = q.cpu().view(torch.float8_e4m3fn).double().view(T, K // 128, 128)
    s = sfa.cpu()[:, :T].t().double()
    assert not sfa.cpu()[:, T:].any()
    cells, ctol = ref.view(T, -1, 128), tol.view(T, -1, 128)
    amax, atol = cells.abs().amax(2), ctol.amax(2)
    assert ((s - amax / 448).abs() <= (atol + 2 * U * amax) / 448).all()
    # a code is within half a step of the value it stands for: 2^-4 of it, or 2^-10 among the subnormals
    err = (code * s.unsqueeze(2) - cells).abs()
    bound = torch.maximum(2.0 ** -4 * (cells.abs() + ctol), 2.0 ** -10 * s.unsqueeze(2)) + ctol + 4 * U * cells.abs()
    assert (err <= bound).all()
    if xt == torch.float32:   # the fp32 result is not rounded before the cast: the same scales and codes
        y = ops.layer_norm(cuda(x), cuda(w), cuda(b), rms=rms).cpu().view(T, -1, 128)
        sc = y.abs().amax(2) / 448
        assert torch.equal(sc, sfa.cpu()[:, :T].t())
        assert torch.equal((y / sc.unsqueeze(2)).view(T, K).to(torch.float8_e4m3fn).view(torch.uint8), q.cpu())


@pytest.mark.parametrize("T,K", [(7, 384), (333, 384), (333, 2048)])
def test_result_and_cast_in_one_call(T, K):
    x, w, b = make(T, K, torch.bfloat16, torch.bfloat16, False, seed=9)
    x, w, b = cuda(x), cuda(w), cuda(b)
    y, mean, rstd = ops.layer_norm(x, w, b, stats=True)
    q, sfa = ops.layer_norm_cast(x, w, b)
    y2, q2, sfa2 = torch.empty_like(y), torch.empty_like(q), torch.zeros_like(sfa)
    _lib.dg_layer_norm(x, w, b, y2, q2, sfa2, None, None, T, K, 1e-5, 0, 0, 0)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(sfa, sfa2)


@pytest.mark.parametrize("T,K", [(6, 520), (320, 520), (320, 1024), (320, 333), (320, 96)])
@pytest.mark.parametrize("rms", [False, True])
def test_bad_rows_stay_alone(T, K, rms):
    """NaN, infinity and the lowest value in some rows leave every other row's bits as they were."""
    x, w, b = make(T, K, torch.float32, torch.float32, rms, seed=10)
    dy = torch.randn(T, K, generator=torch.Generator().manual_seed(3))
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[1, 2, T - 1]] = True
    xb = x.clone()
    xb[1, 3], xb[2, K - 1], xb[T - 1, 0] = float("nan"), float("inf"), -3.4e38
    outs = []
    for v in (x, xb):
        y, mean, rstd = ops.layer_norm(cuda(v), cuda(w), cuda(b), rms=rms, stats=True)
        dx = ops.layer_norm_backward(cuda(dy), cuda(v), cuda(w), mean, rstd, bias=not rms, rms=rms)[0]
        outs.append([t.cpu()[~bad] for t in (y, rstd, dx)])
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_cast_of_zero_rows():
    q, sfa = ops.layer_norm_cast(torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda"))
    assert not q.any() and (sfa[:, :3] == 1).all()


def ref_backward(dy, x, w, mean, rstd, rms):
    """Gradients from the fp32 statistics, and their tolerances."""
    dy, x = dy.double(), x.double()
    mu = 0 if rms else mean.double()[:, None]
    r = rstd.double()[:, None]
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    xh, uu = (x - mu) * r, dy * w
    c1 = 0 if rms else uu.mean(1, keepdim=True)
    c2 = (uu * xh).mean(1, keepdim=True)
    dx = r * (uu - c1 - xh * c2)
    a1, a2 = uu.abs().mean(1, keepdim=True), (uu * xh).abs().mean(1, keepdim=True)
    tol = 80 * U * r * (uu.abs() + (0 if rms else a1) + xh.abs() * a2)
    # a column's sum over T rows: at most T - 1 additions one after another, 8 roundings a term
    return dx, tol, (dy * xh).sum(0), (x.shape[0] + 8) * U * (dy * xh).abs().sum(0), dy.sum(0), \
        (x.shape[0] + 8) * U * dy.abs().sum(0)


@pytest.mark.parametrize("T,K", SHAPES + [(2000, 512), (1111, 7168), (5000, 40), (4000, 33)])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [False, True])
def test_backward(T, K, xt, rms):
    for wt, weight, bias in ((torch.float32, True, True), (torch.bfloat16, True, False), (torch.bfloat16, False, True)):
        x, w, _ = make(T, K, xt, wt, rms, seed=3, weight=weight)
        dy = torch.randn(T, K, generator=torch.Generator().manual_seed(T + K)).to(xt)
        _, mu, r, _ = ref_forward(x, w, None, 1e-5, rms)
        mean, rstd = None if rms else mu.float(), r.float()
        dx, dw, db = ops.layer_norm_backward(cuda(dy), cuda(x), cuda(w), cuda(mean), cuda(rstd), bias=bias and not rms,
                                             rms=rms)
        rx, tx, rw, tw, rb, tb = ref_backward(dy, x, w, mean, rstd, rms)
        assert dx.dtype == xt and ((dx.cpu().double() - rx).abs() <= tx + STEP[xt] * (rx.abs() + tx)).all()
        assert (dw is not None) == weight and (db is not None) == (bias and not rms)
        if weight:
            assert ((dw.cpu().double() - rw).abs() <= tw).all()
        if db is not None:
            assert ((db.cpu().double() - rb).abs() <= tb).all()


@pytest.mark.parametrize("rms", [False, True])
def test_backward_against_differences(rms):
    """The directional derivative of sum(y·dy) along v, from the kernels' gradients and from central
    differences of the 64-bit forward. The second carries an error of h^2; the first one the
    tolerances above, summed over the elements."""
    T, K, h = 6, 96, 1e-5
    x, w, b = make(T, K, torch.float32, torch.float32, rms, seed=4)
    g = torch.Generator().manual_seed(5)
    dy, vx, vw, vb = (torch.randn(s, generator=g) for s in ((T, K), (T, K), (K,), (K,)))
    _, mean, rstd = ops.layer_norm(cuda(x), cuda(w), cuda(b), rms=rms, stats=True)
    dx, dw, db = ops.layer_norm_backward(cuda(dy), cuda(x), cuda(w), mean, rstd, bias=not rms, rms=rms)

    def f(s):
        bb = None if rms else b.double() + s * vb.double()
        y = ref_forward(x.double() + s * vx.double(), w.double() + s * vw.double(), bb, 1e-5, rms)[0]
        return float((y * dy.double()).sum())
    num = (f(h) - f(-h)) / (2 * h)
    got = float((dx.cpu().double() * vx).sum() + (dw.cpu().double() * vw).sum())
    if not rms:
        got += float((db.cpu().double() * vb).sum())
    rx, tx, _, tw, _, tb = ref_backward(dy, x, w, None if rms else mean.cpu(), rstd.cpu(), rms)
    # the statistics' own error (80u of r, twice over in the products) moves dx by as much again
    allow = float((3 * tx * vx.abs()).sum() + (3 * tw * vw.abs()).sum() + (tb * vb.abs()).sum())
    curve = 1e-6 * abs(num) + 1e-6   # h^2 = 1e-10 times third derivatives, and 1e-16/h of the differences
    assert abs(got - num) <= allow + curve


def test_same_bits_every_time_on_streams_and_in_graphs():
    x, w, b = make(700, 1536, torch.bfloat16, torch.float32, False, seed=6)
    dy = torch.randn(700, 1536, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x, w, b, dy = (t.cuda() for t in (x, w, b, dy))

    def step(stream=None):
        y, mean, rstd = ops.layer_norm(x, w, b, stats=True, stream=stream)
        return (y, *ops.layer_norm_backward(dy, x, w, mean, rstd, stream=stream), *ops.layer_norm_cast(x, w, b, stream=stream))
    ref = step()
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = step(s)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for graph, out in graphs + graphs:
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, ref))


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(256, device="cuda")
    s = torch.zeros(4, device="cuda")
    for call in (lambda: ops.layer_norm(x.t()), lambda: ops.layer_norm(x.half()), lambda: ops.layer_norm(x[0]),
                 lambda: ops.layer_norm(x, w[:128]), lambda: ops.layer_norm(x, w.double()), lambda: ops.layer_norm(x, w, rms=True, bias=w),
                 lambda: ops.layer_norm(x, w, w.bfloat16()), lambda: ops.layer_norm(x, out=x.float()),
                 lambda: ops.layer_norm_cast(x[:, :200].contiguous()), lambda: ops.layer_norm_backward(x.float(), x, w, s, s),
                 lambda: ops.layer_norm_backward(x, x, w, None, s), lambda: ops.layer_norm_backward(x, x, w, s, s[:2]),
                 lambda: ops.layer_norm_backward(x, x, w, None, s, rms=True, bias=True)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(_lib.DgError):
        ops.layer_norm(torch.zeros(1, 40000, device="cuda"))
    with pytest.raises(_lib.DgError):
        ops.layer_norm(x, eps=-1.0)
    with pytest.raises(_lib.DgError) as e:
        ops.layer_norm(torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:260].view(4, 64))
    assert e.value.status == _lib.DG_ERR_ALIGNMENT


def test_more_than_2_to_31_elements():
    """Offsets that pass 32 bits: 270000 rows of 8192, the last ones compared with the same rows alone."""
    T, K = 270000, 8192
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    last, w, b = make(5, K, torch.bfloat16, torch.float32, False, seed=11)
    x[-5:] = cuda(last)
    y, mean, rstd = ops.layer_norm(x, cuda(w), cuda(b), stats=True)
    ref, mu, r, tol = ref_forward(last, w, b, 1e-5, False)
    assert ((y[-5:].cpu().double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all()
    assert torch.equal(y[0], cuda(b).bfloat16()) and torch.equal(y[T // 2], y[0])
    dy = torch.zeros_like(x)
    dl = torch.randn(5, K, generator=torch.Generator().manual_seed(4)).bfloat16()
    dy[-5:] = cuda(dl)
    dx, dw, db = ops.layer_norm_backward(dy, x, cuda(w), mean, rstd)
    rx, tx, rw, tw, rb, tb = ref_backward(dl, last, w, mean[-5:].cpu(), rstd[-5:].cpu(), False)
    assert ((dx[-5:].cpu().double() - rx).abs() <= tx + 2.0 ** -8 * (rx.abs() + tx)).all()
    assert not dx[:T - 5].any()
    assert ((dw.cpu().double() - rw).abs() <= tw).all() and ((db.cpu().double() - rb).abs() <= tb).all()


@pytest.mark.parametrize("K", [200, 768, 1000, 1001, 7168, 8191, 12288, 12296])
@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_rows_of_one_value_have_no_deviation(T, K, xt):
    """Rows of one value: its mean is the value, its deviation 0 and the result the bias, exactly, however many rows
    share the call. The values have 8 bits at most and K <= 2^14, so every sum of them is exact in fp32."""
    values = torch.tensor([3.0, 1000.0, -49920.0, 0.375]).repeat(T // 4)
    x = values[:, None].expand(T, K).to(xt).contiguous()
    _, w, b = make(1, K, xt, torch.float32, False, seed=12)
    y, mean, rstd = ops.layer_norm(cuda(x), cuda(w), cuda(b), stats=True)
    assert torch.equal(mean.cpu(), values)
    assert ((rstd.cpu().double() - 1e-5 ** -0.5).abs() <= 4 * U * 1e-5 ** -0.5).all()   # eps and the root: 2 ulp
    assert torch.equal(y.cpu(), b.to(xt).expand(T, K))
    if K % 128 == 0:
        q, sfa = ops.layer_norm_cast(cuda(x))
        assert not q.any() and (sfa[:, :T] == 1).all()


@pytest.mark.parametrize("K", [200, 768, 1000, 1001, 7168, 8191, 12288, 20001])
@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_equal_gradients_of_equal_values_cancel(T, K, xt):
    """dy of one value in a row of one value: u is its own mean and xh is 0, so dx is 0 and not r times an ulp of u.
    The values have 8 bits at most and K < 2^15, so every sum of them is exact in fp32."""
    x = torch.tensor([3.0, 1000.0, -49920.0, 0.375]).repeat(T // 4)
    dy = torch.tensor([1.0, 3.0, -125.0, 0.375]).repeat(T // 4)
    rstd = torch.full((T,), 316.0)
    rows = [v[:, None].expand(T, K).to(xt).contiguous() for v in (dy, x)]
    dx, _, db = ops.layer_norm_backward(cuda(rows[0]), cuda(rows[1]), None, cuda(x), cuda(rstd))
    assert not dx.any()
    assert torch.equal(db.cpu(), dy.sum().expand(K))


def test_two_graphs_share_the_backward_workspace():
    """Two graphs captured on one memory pool: the backward pass's workspace of the first is free again when the second is
    captured, so both may use the same memory. Replayed in any order, each gives the eager bits."""
    x, w, b = (t.cuda() for t in make(700, 1536, torch.bfloat16, torch.float32, False, seed=14))
    dys = [torch.randn(700, 1536, generator=torch.Generator().manual_seed(s)).bfloat16().cuda() for s in (1, 2)]
    _, mean, rstd = ops.layer_norm(x, w, b, stats=True)
    refs = [ops.layer_norm_backward(dy, x, w, mean, rstd) for dy in dys]
    torch.cuda.synchronize()
    pool, graphs = None, []
    for dy in dys:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = ops.layer_norm_backward(dy, x, w, mean, rstd)
        pool = graph.pool()
        graphs.append((graph, out))
    for i in (0, 1, 1, 0, 0, 1):
        for o in graphs[i][1]:
            o.zero_()
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(graphs[i][1], refs[i]))
