"""Refusals of the router, the experts' layer and the draw of a token: status codes of the C
entry points and the binding's own checks. Nothing reaches a GPU."""

import ctypes

import pytest
import torch

import w4a16_int4_weight_amd as w

P = 0x1000        # an aligned address that no refused call looks at


def route(x=P, router=P, bias=None, dtype=1, M=4, K=256, E=8, T=2, score=0, normalize=1, scale=1.0, ids=P, weights=P, ws=P, ws_bytes=1 << 30):
    return w.lib.w4a16_route(x, router, bias, dtype, M, K, E, T, score, normalize, scale, ids, weights, ws, ws_bytes, None)


def moe(x=P, ids=P, weights=P, up=P, up_bytes=1 << 40, up_stride=1 << 20, down=P, down_bytes=1 << 40, down_stride=1 << 20, dtype=1, residual=None,
        y=P, M=4, K=256, F=128, E=8, T=2, G=128, act=0, ws=P, ws_bytes=1 << 40):
    return w.lib.w4a16_moe(x, ids, weights, up, up_bytes, up_stride, down, down_bytes, down_stride, dtype, residual, y, M, K, F, E, T, G, act,
                           ws, ws_bytes, None)


def layer(router=P, score=0, scale=1.0, E=8, T=2, ids=P, weights=P, M=4, ws_bytes=1 << 40):
    return w.lib.w4a16_moe_layer(P, router, None, score, 1, scale, P, 1 << 40, 1 << 20, P, 1 << 40, 1 << 20, 1, None, ids, weights, P, M, 256, 128,
                                 E, T, 128, 0, P, ws_bytes, None)


def sample(logits=P, kind=1, ld=100, u=P, M=4, V=100, how=True, ids=P, logprob=None, ws=P, ws_bytes=1 << 40, **settings):
    s = w._Sampling(1.0, 0, 1.0, 0.0)
    for k, v in settings.items():
        setattr(s, k, v)
    return w.lib.w4a16_sample(logits, kind, ld, u, M, V, ctypes.byref(s) if how else None, ids, logprob, ws, ws_bytes, None)


NULL, SHAPE, GROUP, DTYPE, ALIGN, SIZE, PATH = 1, 2, 3, 4, 5, 6, 9


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(router=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(ws=None), NULL),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=200), SHAPE), (dict(K=(1 << 20) + 128), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(T=0), SHAPE), (dict(T=9), SHAPE), (dict(E=64, T=33), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(dtype=2), DTYPE), (dict(score=2), PATH), (dict(x=P + 8), ALIGN), (dict(router=P + 2), ALIGN),
    (dict(bias=P + 2), ALIGN), (dict(ids=P + 1), ALIGN), (dict(weights=P + 2), ALIGN), (dict(ws=P + 8), ALIGN), (dict(ws_bytes=511), SIZE)])
def test_route_refusals(kw, code):
    assert route(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(up=None), NULL), (dict(down=None), NULL), (dict(y=None), NULL),
    (dict(ws=None), NULL), (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=200), SHAPE), (dict(F=64), SHAPE), (dict(F=0), SHAPE),
    (dict(F=-128), SHAPE), (dict(F=(1 << 15) + 128), SHAPE), (dict(K=(1 << 15) + 128), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(T=0), SHAPE), (dict(T=33), SHAPE), (dict(G=0), GROUP), (dict(G=256), GROUP), (dict(G=48), GROUP), (dict(dtype=3), DTYPE), (dict(act=3), PATH),
    (dict(x=P + 8), ALIGN), (dict(y=P + 8), ALIGN), (dict(up=P + 4), ALIGN), (dict(down=P + 4), ALIGN), (dict(residual=P + 2), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(weights=P + 2), ALIGN), (dict(up_stride=(1 << 20) + 8), ALIGN), (dict(down_stride=(1 << 20) + 8), ALIGN),
    (dict(ws=P + 8), ALIGN), (dict(up_stride=16), SIZE), (dict(down_stride=16), SIZE), (dict(up_bytes=7 << 20), SIZE), (dict(down_bytes=7 << 20), SIZE),
    (dict(up_bytes=100), SIZE), (dict(ws_bytes=1024), SIZE)])
def test_moe_refusals(kw, code):
    assert moe(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(router=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(score=5), PATH), (dict(scale=float("nan")), SHAPE),
    (dict(T=9), SHAPE), (dict(router=P + 8), ALIGN), (dict(ids=P + 2), ALIGN), (dict(ws_bytes=1024), SIZE)])
def test_layer_refusals(kw, code):
    assert layer(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(u=None), NULL), (dict(ids=None), NULL), (dict(how=False), NULL), (dict(M=-1), SHAPE), (dict(V=0), SHAPE),
    (dict(V=101), SHAPE), (dict(V=(1 << 28) + 1, ld=1 << 29), SHAPE), (dict(ld=(1 << 40) + 1), SHAPE), (dict(kind=3), DTYPE), (dict(kind=-1), DTYPE),
    (dict(logits=P + 1), ALIGN), (dict(kind=2, logits=P + 2), ALIGN), (dict(u=P + 2), ALIGN), (dict(ids=P + 2), ALIGN), (dict(logprob=P + 2), ALIGN),
    (dict(temperatures=P + 2), ALIGN), (dict(top_ks=P + 1), ALIGN), (dict(top_ps=P + 2), ALIGN), (dict(min_ps=P + 2), ALIGN)])
def test_sample_refusals(kw, code):
    assert sample(**kw) == code


def test_no_rows_is_a_valid_call():
    assert route(M=0, x=None, ws=None) == 0
    assert moe(M=0, x=None, ws=None) == 0
    assert layer(M=0, ids=None) == 0
    assert sample(M=0, logits=None, ws=None) == 0


def test_workspaces_of_unsupported_shapes_are_none():
    assert w.w4a16_route_workspace_bytes(4, 200, 8, 2) == 0 and w.w4a16_route_workspace_bytes(0, 256, 8, 2) == 0
    assert w.w4a16_moe_workspace_bytes(4, 256, 64, 8, 2, 128) == 0 and w.w4a16_moe_workspace_bytes(4, 256, 128, 8, 2, 256) == 0
    assert w.w4a16_moe_layer_workspace_bytes(4, 256, 128, 8, 9, 128) == 0
    assert w.w4a16_moe_workspace_bytes(4, 256, 128, 8, 9, 128) > 0
    assert w.w4a16_sample_workspace_bytes(0, 100) == 0 and w.w4a16_sample_workspace_bytes(4, 0) == 0
    # more rows than a pass need no more than a full pass
    full = w.w4a16_moe_workspace_bytes(16384 // 8, 256, 128, 8, 8, 128)
    assert w.w4a16_moe_workspace_bytes(1 << 20, 256, 128, 8, 8, 128) == full


def test_binding_refuses_before_the_library():
    bf = torch.bfloat16
    x, router = torch.zeros((4, 256), dtype=bf), torch.zeros((8, 256), dtype=bf)
    ids, weights = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    up = torch.zeros((8, w.w4a16_packed_bytes(256, 256, 128)), dtype=torch.uint8)
    down = torch.zeros((8, w.w4a16_packed_bytes(128, 256, 128)), dtype=torch.uint8)
    ok = dict(gate_up=up, down=down, F=128)
    for bad in (lambda: w.w4a16_route(x, router.half(), 2), lambda: w.w4a16_route(x, router[:, :128], 2), lambda: w.w4a16_route(x.t(), router, 2),
                lambda: w.w4a16_route(x, router, 2, bias=torch.zeros(7)), lambda: w.w4a16_route(x, router, 2, bias=torch.zeros(8, dtype=bf)),
                lambda: w.w4a16_route(x, router, 2, ids=torch.zeros((4, 3), dtype=torch.int32)),
                lambda: w.w4a16_moe(x, ids.long(), weights, **ok), lambda: w.w4a16_moe(x, ids[:3], weights, **ok),
                lambda: w.w4a16_moe(x, ids, weights.half(), **ok), lambda: w.w4a16_moe(x, ids, weights[:, :1], **ok),
                lambda: w.w4a16_moe(x, ids, weights, up, down[:7], 128), lambda: w.w4a16_moe(x, ids, weights, up.view(torch.int8), down, 128),
                lambda: w.w4a16_moe(x, ids, weights, up[0], down, 128), lambda: w.w4a16_moe(x, ids, weights, up[:, ::2], down, 128),
                lambda: w.w4a16_moe(x, ids, weights, residual=x.half(), **ok), lambda: w.w4a16_moe(x, ids, weights, residual=x[:3], **ok),
                lambda: w.w4a16_moe(x, ids, weights, y=x.half(), **ok),
                lambda: w.w4a16_moe_layer(x, router[:7].contiguous(), up, down, 128, 2),
                lambda: w.w4a16_sample(x.to(torch.float64), torch.zeros(4)), lambda: w.w4a16_sample(x[0], torch.zeros(4)),
                lambda: w.w4a16_sample(x[:, ::2], torch.zeros(4)), lambda: w.w4a16_sample(x, torch.zeros(3)),
                lambda: w.w4a16_sample(x, torch.zeros(4, dtype=torch.float64)), lambda: w.w4a16_sample(x, torch.zeros(4), top_k=torch.zeros(4)),
                lambda: w.w4a16_sample(x, torch.zeros(4), top_p=torch.zeros(5)), lambda: w.w4a16_sample(x.expand(4, 256)[:1].expand(4, 256), torch.zeros(4)),
                lambda: w.w4a16_sample(x, torch.zeros(4), ids=torch.zeros(4)),
                # tensors that are not on a GPU
                lambda: w.w4a16_route(x, router, 2), lambda: w.w4a16_moe(x, ids, weights, **ok), lambda: w.w4a16_sample(x, torch.zeros(4))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(w.W4A16Error):
        w.w4a16_route(x, router, 2, score="relu")
    with pytest.raises(w.W4A16Error):
        w.w4a16_route(x, router, 0)
    with pytest.raises(w.W4A16Error):
        w.w4a16_moe(x, ids, weights, act="relu", **ok)
