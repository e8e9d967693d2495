"""Argument checks of the operators around the experts' products (norm, routing, layouts, top-k dispatch,
combine): everything the host can refuse is refused before any device is asked for."""
import pytest
import torch

from moe_grouped_gemm_sm_b200 import _lib, build, ops

P = 16            # a non-null, aligned address that nothing reads
BAD, ALIGN, OK = _lib.DG_ERR_INVALID_ARG, _lib.DG_ERR_ALIGNMENT, _lib.DG_OK
BF16, FP32, SOFTMAX, SIGMOID = 0, 1, 0, 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("change,status", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(q=P), BAD), (dict(sfa=P), BAD), (dict(T=-1), BAD), (dict(K=0), BAD),
    (dict(K=32769), BAD), (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(rms=1), BAD), (dict(x_type=2), BAD),
    (dict(w_type=-1), BAD), (dict(q=P, sfa=P, K=100), BAD), (dict(x=P + 4), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(b=P + 2), ALIGN), (dict(y=P + 8), ALIGN), (dict(q=P + 8, sfa=P), ALIGN), (dict(T=0), OK)])
def test_norm(lib, change, status):
    a = dict(x=P, w=P, b=P, y=P, q=None, sfa=None, mean=P, rstd=P, T=4, K=128, eps=1e-5, rms=0, x_type=BF16, w_type=BF16)
    a.update(change)
    assert lib.dg_layer_norm(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(rstd=None), BAD), (dict(dx=None), BAD), (dict(ws=None), BAD),
    (dict(wb=100), BAD), (dict(T=-1), BAD), (dict(K=0), BAD), (dict(K=32769), BAD), (dict(x_type=7), BAD),
    (dict(dx=P + 4), ALIGN), (dict(dw=P + 4), ALIGN), (dict(ws=P + 8), ALIGN), (dict(T=0, dw=None, db=None), OK)])
def test_norm_backward(lib, change, status):
    a = dict(dy=P, x=P, w=P, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P, wb=1 << 30, T=4, K=128, x_type=FP32, w_type=FP32)
    a.update(change)
    assert lib.dg_layer_norm_backward(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), BAD), (dict(ids=None), BAD), (dict(w=None), BAD), (dict(T=-1), BAD), (dict(E=0), BAD),
    (dict(E=1025, groups=1, topk_groups=1), BAD), (dict(k=0), BAD), (dict(k=33), BAD), (dict(E=8, k=9), BAD),
    (dict(groups=0), BAD), (dict(groups=7), BAD), (dict(E=1024, groups=64), BAD), (dict(topk_groups=0), BAD),
    (dict(topk_groups=9), BAD), (dict(group_top=0), BAD), (dict(group_top=3), BAD), (dict(score=2), BAD),
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(dtype=2), BAD), (dict(logits=P + 2), ALIGN),
    (dict(ids=P + 4), ALIGN), (dict(T=0), OK)])
def test_route(lib, change, status):
    a = dict(logits=P, bias=P, ids=P, w=P, T=4, E=64, k=8, groups=8, topk_groups=4, group_top=2, score=SIGMOID, renorm=1,
             scale=1.0, dtype=BF16)
    a.update(change)
    assert lib.dg_moe_route(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(gw=None), BAD), (dict(logits=None), BAD), (dict(ids=None), BAD), (dict(g=None), BAD), (dict(E=1025), BAD),
    (dict(k=33), BAD), (dict(k=65), BAD), (dict(score=-1), BAD), (dict(scale=NAN), BAD), (dict(dtype=5), BAD),
    (dict(g=P + 8), ALIGN), (dict(T=0), OK)])
def test_route_backward(lib, change, status):
    a = dict(gw=P, logits=P, ids=P, g=P, T=4, E=64, k=8, score=SOFTMAX, renorm=0, scale=1.0, dtype=FP32)
    a.update(change)
    assert lib.dg_moe_route_backward(*a.values(), None) == status


def test_layouts(lib):
    def contiguous(ids=P, dst=P, layout=P, ks=P, T=4, k=2, G=8, M=1024):
        return lib.dg_moe_layout_contiguous(ids, dst, layout, ks, T, k, G, M, None)

    def masked(ids=P, dst=P, mm=P, T=4, k=2, G=8, M=256):
        return lib.dg_moe_layout_masked(ids, dst, mm, T, k, G, M, None)

    for bad in (dict(ids=None), dict(dst=None), dict(layout=None), dict(T=-1), dict(k=0), dict(G=0), dict(G=1025),
                dict(M=100), dict(M=-128), dict(T=1 << 30)):
        assert contiguous(**bad) == BAD, bad
    for bad in (dict(ids=None), dict(dst=None), dict(mm=None), dict(T=-1), dict(k=0), dict(G=0), dict(G=1025), dict(M=-1),
                dict(G=1024, M=1 << 21)):
        assert masked(**bad) == BAD, bad
    assert contiguous(layout=P + 4) == ALIGN and contiguous(ks=P + 4) == ALIGN and masked(ids=P + 4) == ALIGN


def test_workspace_sizes(lib):
    assert _lib.dg_layer_norm_backward_workspace(0, 128) == 0
    assert _lib.dg_layer_norm_backward_workspace(1, 128) > 0
    assert _lib.dg_layer_norm_backward_workspace(8192, 7168) <= 64 << 20


def test_dispatch(lib):
    def call(x=P, dst=P, q=P, sfa=P, T=4, k=2, G=8, M=64, K=256):
        return lib.dg_cast_fp8_per_token_scatter_topk(x, dst, q, sfa, T, k, G, M, K, None)

    for bad in (dict(x=None), dict(dst=None), dict(q=None), dict(sfa=None), dict(T=-1), dict(k=0), dict(G=0), dict(M=-1),
                dict(K=0), dict(K=200), dict(G=1 << 16, M=1 << 16), dict(T=1 << 30)):
        assert call(**bad) == BAD, bad
    assert call(x=P + 2) == ALIGN and call(q=P + 8) == ALIGN and call(sfa=P + 4) == ALIGN
    assert call(T=0) == OK and call(M=0) == OK


def test_combine(lib):
    def call(d=P, dst=P, w=P, c=P, y=P, T=4, k=2, N=64, R=512):
        return lib.dg_moe_combine(d, dst, w, c, y, T, k, N, R, None)

    for bad in (dict(d=None), dict(dst=None), dict(y=None), dict(T=-1), dict(k=0), dict(k=33), dict(N=0), dict(N=12),
                dict(R=-1)):
        assert call(**bad) == BAD, bad
    assert call(d=P + 8) == ALIGN and call(c=P + 2) == ALIGN and call(y=P + 2) == ALIGN
    assert call(T=0) == OK

    def back(gy=P, d=P, dst=P, w=P, layout=P, gd=P, gw=P, T=4, k=2, N=64, R=512):
        return lib.dg_moe_combine_backward(gy, d, dst, w, layout, gd, gw, T, k, N, R, None)

    for bad in (dict(gy=None), dict(dst=None), dict(gd=None, gw=None, layout=None), dict(gd=None), dict(d=None),
                dict(T=-1), dict(k=0), dict(k=33), dict(N=20), dict(R=-1)):
        assert back(**bad) == BAD, bad
    assert back(gy=P + 2) == ALIGN and back(gd=P + 2) == ALIGN and back(d=P + 2) == ALIGN


def test_host_tensors_are_refused():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    w = torch.zeros(4, 2)
    for call in (lambda: ops.layer_norm(x), lambda: ops.layer_norm_cast(x),
                 lambda: ops.layer_norm_backward(x, x, None, w[:, 0], w[:, 0]), lambda: ops.moe_route(w, 1),
                 lambda: ops.moe_route_backward(w, w, i), lambda: ops.moe_layout_contiguous(i, 4),
                 lambda: ops.moe_layout_masked(i, 4, 8), lambda: ops.cast_per_token_scatter_topk(x, i, 128),
                 lambda: ops.moe_combine(x, i), lambda: ops.moe_combine_backward(x, x, i)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_sizes_that_do_not_fit_the_abi_are_refused():
    with pytest.raises(ValueError, match="32 bits"):
        ops._check_sizes(5, 2 ** 31)
    with pytest.raises(ValueError, match="32 bits"):
        ops._check_sizes(-2 ** 31 - 1)
    ops._check_sizes(0, -1, 2 ** 31 - 1)
