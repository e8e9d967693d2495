"""Routing to experts and its gradient against the definition in 64 bits.

The choice is compared exactly. Weights: expf is within 2 units in the last place (4u, u = 2^-24),
its argument x - max is rounded by u·|x - max|, a sum of up to 1024 scores takes 32 + 5 additions, the
quotients and the scale round once each: within (64 + max|x - max|)·u of the weight."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_sm_b200 import _lib, build, ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FMAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def reference(x, bias, k, groups, topk_groups, group_top, score, renorm, scale):
    """ids [T,k], weights [T,k] and the row's spread of logits, token by token from the definition."""
    T, E = x.shape
    ids, w, spread = np.full((T, k), -1, np.int32), np.zeros((T, k)), np.zeros((T, 1))
    for t in range(T):
        xt = np.minimum(np.where(np.isnan(x[t]), -np.inf, x[t]).astype(np.float64), FMAX)
        on = xt > -np.inf
        if not on.any():
            continue
        if score == "softmax":
            e = np.where(on, np.exp(np.where(on, xt, 0) - xt.max()), 0)
            s = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s = np.where(on, np.where(xt >= 0, 1 / (1 + np.exp(-np.abs(xt))), np.exp(-np.abs(xt)) / (1 + np.exp(-np.abs(xt)))), 0)
        b = np.zeros(E) if bias is None else bias.astype(np.float64)
        c = [(s[e] + b[e], xt[e] if bias is None else 0.0) if on[e] and b[e] > -np.inf else None for e in range(E)]
        kept = list(range(groups))
        if groups > 1:
            gs, val = E // groups, []
            for g in range(groups):
                best = sorted((v for v in c[g * gs:(g + 1) * gs] if v is not None), reverse=True)[:group_top]
                one = 1 if group_top == 1 and bias is None else 0   # the largest logit alone decides
                val.append(sum(v[one] for v in best) if best else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-val[g], g))[:topk_groups]
        gs = E // groups
        pool = [e for e in range(E) if c[e] is not None and e // gs in kept]
        # without a bias the logit decides between scores that 64 bits cannot tell apart
        key = (lambda e: (-c[e][0], e)) if bias is not None else (lambda e: (-c[e][1], e))
        chosen = sorted(pool, key=key)[:k]
        ids[t, :len(chosen)] = chosen
        if chosen:
            xs = xt[chosen]
            spread[t] = min(xt.max() - xs.min(), 1e4)
            if score == "softmax":
                v = np.exp(xs - xs.max()) if renorm else s[chosen]
            else:
                m = min(xs.max(), 0.0) if renorm else 0.0
                v = np.where(xs >= 0, 1 / (1 + np.exp(-np.abs(xs))), np.exp(np.minimum(xs - m, 0)) / (1 + np.exp(-np.abs(xs))))
            w[t, :len(chosen)] = (v / v.sum() if renorm else v) * scale
    return ids, w, spread


def check(x, bias, k, groups=1, topk_groups=1, group_top=1, score="softmax", renorm=True, scale=1.0):
    kw = dict(bias=None if bias is None else bias.cuda(), groups=groups, topk_groups=topk_groups, group_top=group_top,
              score=score, renorm=renorm, scale=scale)
    w, ids = ops.moe_route(x.cuda(), k, **kw)
    ri, rw, spread = reference(x.float().numpy(), None if bias is None else bias.numpy(), k, groups, topk_groups, group_top,
                               score, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), ri)
    tiny = 2.0 ** -125 * abs(scale)   # an fp32 score below 2^-126 keeps an absolute step only
    tol = (64 + spread) * U * np.abs(rw) + tiny
    assert (np.abs(w.cpu().numpy().astype(np.float64) - rw) <= tol).all()
    # the same rows again and again: many tokens take another form of the kernel
    n = 1030 // x.shape[0] + 1
    wn, idn = ops.moe_route(x.cuda().repeat(n, 1), k, **kw)
    assert np.array_equal(idn.cpu().numpy(), np.tile(ri, (n, 1)))
    assert (np.abs(wn.cpu().numpy().astype(np.float64) - np.tile(rw, (n, 1))) <= np.tile(tol, (n, 1))).all()
    return w, ids


def logits(T, E, dtype, seed=0, sigma=1.5):
    g = torch.Generator().manual_seed(seed * 1009 + T * 7 + E)
    return (sigma * torch.randn(T, E, generator=g)).to(dtype), 0.1 * torch.randn(E, generator=g)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 5, 3), (9, 31, 31), (7, 33, 32), (64, 64, 6), (130, 160, 6),
                                   (33, 256, 8), (11, 300, 8), (4, 512, 17), (6, 1024, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_and_weights(T, E, k, dtype, score):
    x, b = logits(T, E, dtype)
    for bias in (None, b):
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            check(x, bias, k, score=score, renorm=renorm, scale=scale)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("E,groups,topk_groups,k", [(256, 8, 4, 8), (64, 8, 3, 6), (128, 8, 4, 4), (256, 8, 1, 8), (96, 3, 2, 7), (384, 8, 1, 8), (40, 20, 5, 10),
                                                    (32, 32, 9, 9), (1024, 32, 8, 16), (100, 4, 4, 5)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, groups, topk_groups, k, group_top, score):
    for dtype in (torch.bfloat16, torch.float32):
        x, b = logits(67, E, dtype, seed=groups)
        for bias in (None, b):
            check(x, bias, k, groups, topk_groups, group_top, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_extreme_logits(score):
    inf, low = float("inf"), -FMAX
    x, b = logits(12, 48, torch.float32, seed=9)
    x[0] = -inf                                   # nothing left
    x[1] = -inf
    x[1, 17] = 0.25                               # one expert left
    x[2, 8:] = -inf                               # k - 2 left
    x[3] = low                                    # the lowest value is a value
    x[4, ::2] = low
    x[5] = 7.0                                    # all equal: in the order of the index
    x[6, 3] = inf
    x[7, 5] = x[7, 40] = inf                      # both count as the largest value
    x[8] = -90.0 + x[8]                           # sigmoid far below one
    x[9] = x[9] * 40
    x[10] = -300.0 - torch.arange(48.0)
    for bias in (None, b):
        for groups, kept in ((1, 1), (6, 2)):
            for top in (1, 2):
                for renorm in (True, False):
                    check(x, bias, 10, groups, kept, top, score, renorm)
    b2 = b.clone()
    b2[::3] = -inf                                # experts switched off by the bias
    check(x, b2, 10, score=score)
    check(x, b2, 10, 6, 2, 2, score=score)
    assert _lib.dg_get_device_error() == _lib.DG_OK
    x[11, 4] = float("nan")
    check(x, None, 10, score=score)
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
    b2[7] = float("nan")
    b3 = b2.clone()
    b3[7] = -inf
    x = x[:9]
    w, ids = ops.moe_route(x.cuda(), 10, bias=b2.cuda(), score=score)
    w3, ids3 = ops.moe_route(x.cuda(), 10, bias=b3.cuda(), score=score)
    assert torch.equal(ids, ids3) and torch.equal(w, w3)
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_next_to_each_other(score):
    """Choice values that differ by less than an fp32 rounding (a few 1e-10) and ones that are equal: the real
    order decides, then the index. 64 bits hold the difference with room (1e-16)."""
    g = torch.Generator().manual_seed(3)
    T, E = 256, 64
    x = torch.randn(T, E, generator=g).clamp(-2, 2)
    x[:, 32:] = torch.nextafter(x[:, :32], torch.where(torch.rand(T, 32, generator=g) < 0.5, -9.0, 9.0))
    x[: T // 4, 32:] = x[: T // 4, :32]
    b = 0.05 * torch.randn(E, generator=g)
    b[32:] = b[:32]
    for groups, kept, top in ((1, 1, 1), (2, 1, 1), (8, 4, 2), (16, 5, 2)):
        check(x, b, 8, groups, kept, top, score)
        check(x, torch.zeros(E), 8, groups, kept, top, score)
        check(x, None, 8, groups, kept, top, score)
    y = x.bfloat16()                              # many equal logits
    check(y, b, 8, score=score)
    check(y, None, 8, 8, 4, 2, score=score)
    check(y, torch.zeros(E), 8, 8, 4, 1, score=score)
    big = 1000.0 + b                              # a bias that leaves the score few bits
    check(x, big, 8, score=score)
    check(x, big, 8, 8, 4, 2, score=score)


def ref_weights(x, ids, score, renorm, scale):
    """The weights of a given choice as a differentiable function of 64-bit logits."""
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    on = ids >= 0
    v = s.gather(1, ids.clamp(min=0).long()) * on
    return (v / v.sum(1, keepdim=True).clamp(min=1e-300) if renorm else v) * scale


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 5, 3), (9, 31, 31), (7, 33, 32), (64, 64, 6), (33, 256, 8), (6, 1000, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient(T, E, k, dtype, score, renorm):
    x, _ = logits(T, E, dtype, seed=4)
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    _, ids = ops.moe_route(x.cuda(), k, score=score, renorm=renorm)
    ids = ids.clone()
    ids[0, k // 2:] = -1                          # a row with fewer choices
    if T > 2:
        ids[2] = -1                               # and one with none
    if T > 3 and k > 1:
        ids[3, 1] = ids[3, 0]                     # the same index twice
    got = ops.moe_route_backward(g.cuda(), x.cuda(), ids, score=score, renorm=renorm, scale=2.5)
    xd = x.double().requires_grad_()
    w = ref_weights(xd, ids.cpu(), score, renorm, 2.5)
    (ref,) = torch.autograd.grad((w * g.double()).sum(), xd)
    # each weight within 64u + spread, the sums of k products within another k + 5
    size = (w.detach() * g.double()).abs().sum(1, keepdim=True)
    s = torch.softmax(xd.detach(), 1) if score == "softmax" and not renorm else torch.zeros_like(ref)
    chosen = torch.zeros_like(ref).scatter_add_(1, ids.cpu().clamp(min=0).long(), (w.detach() * g.double()).abs() * (ids.cpu() >= 0))
    share = torch.zeros_like(ref).scatter_add_(1, ids.cpu().clamp(min=0).long(), w.detach().abs() * (ids.cpu() >= 0)) / 2.5
    spread = (xd.detach().amax(1) - xd.detach().amin(1))[:, None]
    # the reference's own rounding: autograd leaves about 1e-18 where the terms of a logit that is not chosen
    # cancel (the kernel writes the exact 0). Those are sums of at most E + k terms of |g·w| <= size, each
    # rounded in 64 bits: (E + k)·2^-53·size
    tol = (2 * (64 + spread) + k + 8) * U * (chosen + size * (share + s)) + (E + k) * 2.0 ** -53 * size
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert got.dtype == dtype and ((got.cpu().double() - ref).abs() <= tol + half * (ref.abs() + tol)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    T, E, k, h = 8, 24, 4, 1e-6
    x, _ = logits(T, E, torch.float32, seed=5)
    gen = torch.Generator().manual_seed(6)
    g, v = torch.randn(T, k, generator=gen), torch.randn(T, E, generator=gen)
    _, ids = ops.moe_route(x.cuda(), k, score=score, renorm=renorm)
    got = ops.moe_route_backward(g.cuda(), x.cuda(), ids, score=score, renorm=renorm, scale=1.5)

    def f(s):
        return float((ref_weights(x.double() + s * v.double(), ids.cpu(), score, renorm, 1.5) * g.double()).sum())
    num = (f(h) - f(-h)) / (2 * h)
    # T·E terms of size <= 1.5·|g|·|v| with about 200u each; differences: h^2 and 1e-16/h
    assert abs(float((got.cpu().double() * v.double()).sum()) - num) <= 200 * U * 1.5 * float(g.abs().sum() * v.abs().max()) + 1e-8


def test_backward_refuses_an_id_outside():
    x, _ = logits(4, 16, torch.float32)
    ids = torch.tensor([[1, 16], [2, 3], [-5, 4], [0, 1 << 30]], dtype=torch.int32)
    g = torch.ones(4, 2)
    got = ops.moe_route_backward(g.cuda(), x.cuda(), ids.cuda(), score="sigmoid", renorm=False)
    assert _lib.dg_get_device_error() == _lib.DG_ERR_DEVICE
    inside = torch.where((ids < 0) | (ids >= 16), torch.tensor(-1, dtype=torch.int32), ids)
    assert torch.equal(got, ops.moe_route_backward(g.cuda(), x.cuda(), inside.cuda(), score="sigmoid", renorm=False))
    assert _lib.dg_get_device_error() == _lib.DG_OK


def test_streams_graphs_and_no_tokens():
    x, b = logits(500, 256, torch.bfloat16, seed=7)
    x, b = x.cuda(), b.cuda()
    g = torch.randn(500, 8, device="cuda")

    def step(stream=None):
        w, ids = ops.moe_route(x, 8, bias=b, groups=8, topk_groups=4, group_top=2, score="sigmoid", stream=stream)
        return w, ids, ops.moe_route_backward(g, x, ids, score="sigmoid", stream=stream)
    ref = step()
    torch.cuda.synchronize()
    got = step(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, ref))
    w, ids = ops.moe_route(x[:0], 8)
    assert w.shape == ids.shape == (0, 8)
    assert ops.moe_route_backward(w, x[:0], ids).shape == (0, 256)


def test_refusals():
    x = torch.zeros(4, 16, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    g = torch.zeros(4, 2, device="cuda")
    for call in (lambda: ops.moe_route(x.half(), 2), lambda: ops.moe_route(x[0], 2), lambda: ops.moe_route(x.t(), 2),
                 lambda: ops.moe_route(x, 2, bias=torch.zeros(16, device="cuda").bfloat16()),
                 lambda: ops.moe_route(x, 2, bias=torch.zeros(8, device="cuda")), lambda: ops.moe_route(x, 2, score="relu"),
                 lambda: ops.moe_route_backward(g, x, ids.long()), lambda: ops.moe_route_backward(g[:2], x, ids),
                 lambda: ops.moe_route_backward(g.bfloat16(), x, ids), lambda: ops.moe_route_backward(g, x, ids[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ops.moe_route(x, 17), lambda: ops.moe_route(x, 0), lambda: ops.moe_route(x, 2, groups=3),
                 lambda: ops.moe_route(x, 2, groups=4, topk_groups=5), lambda: ops.moe_route(x, 2, group_top=3),
                 lambda: ops.moe_route(x, 2, scale=float("nan"))):
        with pytest.raises(_lib.DgError):
            call()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,top", [(64, 1, 1, 1), (64, 8, 4, 2), (128, 8, 3, 1), (200, 1, 1, 1), (256, 8, 4, 2), (40, 4, 2, 2), (1024, 1, 1, 1), (128, 4, 2, 1)])
def test_gaps_of_every_size(score, E, groups, topk_groups, top):
    """Neighbouring choice values at distances from 1e-9 to 1e-2, and zeros of both signs: whatever precision the
    first look at a token has, the choice is the definition's."""
    g = torch.Generator().manual_seed(E)
    T, half = 160, E // 2
    x = torch.randn(T, E, generator=g)
    gap = 10.0 ** (-9 + 7 * torch.rand(T, half, generator=g, dtype=torch.float64)) * torch.randn(T, half, generator=g).sign()
    perm = torch.randperm(E, generator=g)
    x[:, perm[half:2 * half]] = (x[:, perm[:half]].double() + gap).float()
    x[:8, ::3] = 0.0
    x[:8, 1::3] = -0.0
    x[8:12] *= 1e-39                              # subnormal logits
    b = 0.1 * torch.randn(E, generator=g)
    b[perm[half:2 * half]] = b[perm[:half]]       # the gap is the logits' alone
    for bias in (b, None, torch.zeros(E)):
        check(x, bias, 8, groups, topk_groups, top, score)
        check(x, bias, 30, groups, topk_groups, top, score)
    b2 = b.clone()
    b2[:3] = float("inf")
    b2[3] = FMAX
    check(x[12:], b2, 8, score=score)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 100, 1024])
def test_many_values_next_to_the_lowest(score, E):
    """More values at and one step above the type's lowest than a warp's lanes hold: their order is that of the
    values, in the logits and in the biases."""
    up = float(np.nextafter(np.float32(-FMAX), np.float32(0)))
    x = torch.full((4, E), -FMAX)
    x[0, E // 2:] = up
    x[1, 1::2] = up
    x[2, 5:] = up
    x[2, 40:43] = 0.5
    x[3, E - 3:] = up
    for k in (1, 8, 30):
        check(x, None, k, score=score)
        check(x[:, :E // 4 * 4].contiguous(), None, k, 4, 2, 1, score)
    y, _ = logits(5, E, torch.float32, seed=21)
    for row in x:
        check(y, row, 8, score=score)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_values_beyond_fp32(score):
    """Two choice values of a group may sum to more than fp32 holds, on either side: the groups keep their order, and
    a group of very low values is not one of no experts."""
    x, _ = logits(40, 32, torch.float32, seed=22)
    for low in ([-3e38, -2e38, -2.5e38, -3.2e38], [3e38, 3.3e38, 2e38, 2.5e38], [-3e38, -3.3e38, 3e38, 1.0],
                [-3.3e38, -3e38, -float("inf"), -float("inf")], [FMAX, -FMAX, FMAX, -FMAX]):
        b = torch.tensor(low).repeat_interleave(8)
        for kept in (1, 2, 3):
            check(x, b, 4, 4, kept, 2, score)
        check(x, b, 8, 8, 3, 2, score)
        check(x.repeat(1, 8), b.repeat(8), 8, 8, 3, 2, score)
    assert _lib.dg_get_device_error() == _lib.DG_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size,spread", [(1000.0, 1e-2), (1000.0, 1e-3), (3e4, 0.1), (1e5, 1.0)])
def test_group_values_that_cancel(score, size, spread):
    """Biases of both signs in a group: each choice value is rounded at the bias's size, while the group's value is
    of the scores' size. The choice is that of the 64-bit values, which hold the scores to 2^-53 of the bias."""
    T, E, G = 20000, 64, 8
    g = torch.Generator().manual_seed(int(size))
    x = 0.3 + spread * torch.randn(T, E, generator=g)
    b = torch.full((E,), -size)
    b[::E // G] = size
    c = (torch.softmax(x.double(), 1) if score == "softmax" else torch.sigmoid(x.double())) + b.double()
    best = c.view(T, G, -1).topk(2, dim=2).values.sum(2)
    # rows whose groups or experts 64 bits cannot tell apart are left out: 4 roundings of the bias between them
    gap = best.sort(1).values.diff(dim=1).amin(1)
    kept = best.topk(4, dim=1).indices
    on = torch.zeros(T, G, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(E // G, 1)
    top = c.masked_fill(~on, -float("inf")).topk(7, dim=1)
    gap = torch.minimum(gap, -top.values.diff(dim=1).amax(1))
    sure = gap > 8 * 2.0 ** -53 * size
    assert sure.float().mean() > 0.98
    for rows in (slice(0, T), slice(0, 60)):
        _, ids = ops.moe_route(x[rows].cuda(), 6, bias=b.cuda(), groups=G, topk_groups=4, group_top=2, score=score)
        assert torch.equal(ids.cpu().long()[sure[rows]], top.indices[rows, :6][sure[rows]])
