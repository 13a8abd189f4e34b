"""The training operators' C ABI on the host: what the header declares is exported and
bound, arguments are refused before any device call, workspaces are sized."""

import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, GROUP, DTYPE, ALIGN, SIZE, DEVICE, PATH = 1, 2, 3, 4, 5, 6, 7, 9
P = lambda v: v  # noqa: E731  (an address that is never read)
BIG = 1 << 60


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "w4a16_train.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(w4a16_[a-z_0-9]+)\s*\(", text)))


def test_declared_exported_bound(w):
    assert declared() == ["w4a16_cross_entropy", "w4a16_cross_entropy_workspace_bytes", "w4a16_distill",
                          "w4a16_distill_workspace_bytes", "w4a16_gated", "w4a16_gated_grad", "w4a16_gated_workspace_bytes",
                          "w4a16_gemm_grad", "w4a16_gemm_grad_workspace_bytes"]
    for name in declared():
        assert hasattr(w.lib, name) and callable(getattr(w, name)), name


def gemm_grad(w, dy=256, packed=512, packed_bytes=BIG, dtype=1, dx=1024, M=4, K=256, N=64, G=128, ws=2048, ws_bytes=BIG):
    return w.lib.w4a16_gemm_grad(dy, packed, packed_bytes, dtype, dx, M, K, N, G, ws, ws_bytes, None)


def gated(w, x=256, packed=512, packed_bytes=BIG, dtype=1, h=1024, M=20, K=1024, F=64, G=128, act=0, ws=2048, ws_bytes=BIG):
    return w.lib.w4a16_gated(x, packed, packed_bytes, dtype, h, M, K, F, G, act, ws, ws_bytes, None)


def gated_grad(w, x=256, dh=768, packed=512, packed_bytes=BIG, dtype=1, dx=1024, M=4, K=256, F=64, G=128, act=0, ws=2048,
               ws_bytes=BIG):
    return w.lib.w4a16_gated_grad(x, dh, packed, packed_bytes, dtype, dx, M, K, F, G, act, ws, ws_bytes, None)


def cross_entropy(w, x=256, labels=128, packed=512, packed_bytes=BIG, dtype=1, M=4, K=256, V=1000, G=128, dloss=None, loss=640,
                  lse=704, dx=None, ws=2048, ws_bytes=BIG):
    return w.lib.w4a16_cross_entropy(x, labels, packed, packed_bytes, dtype, M, K, V, G, dloss, loss, lse, dx, ws, ws_bytes, None)


def distill(w, x=256, ids=128, top=192, packed=512, packed_bytes=BIG, dtype=1, M=4, K=256, V=1000, G=128, T=8, tau=1.0,
            dloss=None, loss=640, lse=704, dx=None, ws=2048, ws_bytes=BIG):
    return w.lib.w4a16_distill(x, ids, top, packed, packed_bytes, dtype, M, K, V, G, T, tau, dloss, loss, lse, dx, ws, ws_bytes,
                               None)


CALLS = [gemm_grad, gated, gated_grad, cross_entropy, distill]


@pytest.mark.parametrize("call", CALLS)
def test_common_refusals(w, call):
    for bad in ({"K": 0}, {"K": 200}, {"K": -128}, {"M": -1}, {"M": 1 << 31}, {"K": 1 << 21}):
        assert call(w, **bad) == SHAPE, bad
    for G in (0, 16, 96, 512, -2):
        assert call(w, G=G, K=256) == GROUP, G
    assert call(w, dtype=2) == DTYPE and call(w, dtype=-1) == DTYPE
    assert call(w, packed=None) == NULL
    assert call(w, packed=520) == ALIGN
    assert call(w, packed_bytes=100) == SIZE
    assert call(w, M=0, packed=None) == 0                       # nothing to do
    if not torch.cuda.is_available():
        assert call(w) == DEVICE                                # everything else in order


@pytest.mark.parametrize("call,names", [
    (gemm_grad, ["dy", "dx"]), (gated, ["x", "h"]), (gated_grad, ["x", "dh", "dx"]),
    (cross_entropy, ["x", "labels", "loss", "lse"]), (distill, ["x", "ids", "top", "loss", "lse"])])
def test_pointers(w, call, names):
    for n in names:
        assert call(w, **{n: None}) == NULL, n
        assert call(w, **{n: 1 + 256}) == ALIGN, n


@pytest.mark.parametrize("call,n", [(gemm_grad, "N"), (gated, "F"), (gated_grad, "F"), (cross_entropy, "V"), (distill, "V")])
def test_columns(w, call, n):
    for v in (0, -8, 12, 1 << 40):
        assert call(w, **{n: v}) == SHAPE, v


def test_own_arguments(w):
    for act in (-1, 3, 1 << 20):
        assert gated(w, act=act) == PATH and gated_grad(w, act=act) == PATH
    for T in (0, -1, 257):
        assert distill(w, T=T) == SHAPE
    for tau in (0.0, -1.0, float("inf"), float("nan")):
        assert distill(w, tau=tau) == SHAPE
    assert cross_entropy(w, dx=8 + 1024) == ALIGN and cross_entropy(w, dloss=2 + 1024) == ALIGN


@pytest.mark.parametrize("call,extra", [(gated_grad, {}), (cross_entropy, {}), (cross_entropy, {"dx": 4096}), (distill, {"dx": 4096})])
def test_workspace(w, call, extra):
    assert call(w, ws=None, **extra) == NULL
    assert call(w, ws=2056, **extra) == ALIGN
    assert call(w, ws_bytes=64, **extra) == SIZE


def test_workspace_bytes(w):
    # nothing for what is not supported or needs none
    assert w.w4a16_gemm_grad_workspace_bytes(0, 256, 64, 128) == 0
    assert w.w4a16_gemm_grad_workspace_bytes(4, 250, 64, 128) == 0
    assert w.w4a16_gated_workspace_bytes(4, 256, 12, 128) == 0
    assert w.w4a16_gated_workspace_bytes(1, 2048, 6656, 128) == 0
    assert w.w4a16_cross_entropy_workspace_bytes(4, 256, 1000, 96) == 0
    assert w.w4a16_distill_workspace_bytes(4, 256, 1000, 128, 257) == 0
    # bounded over M: rows go in passes, the vocabulary in pieces of at most 256 MiB
    one = w.w4a16_cross_entropy_workspace_bytes(4096, 2048, 131072, 128, True)
    assert w.w4a16_cross_entropy_workspace_bytes(40960, 2048, 131072, 128, True) == one < 512 << 20
    many = w.w4a16_gated_workspace_bytes(8192, 2048, 6656, 128, True)
    assert w.w4a16_gated_workspace_bytes(81920, 2048, 6656, 128, True) == many < 1 << 30
    for M in (1, 16, 17, 333, 4096):
        plain = w.w4a16_cross_entropy_workspace_bytes(M, 1024, 32008, 64)
        assert 0 < plain <= w.w4a16_cross_entropy_workspace_bytes(M, 1024, 32008, 64, True)


def test_wrappers_refuse(w):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    packed = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        w.w4a16_gated(x.t(), packed, 64)                        # not contiguous
    with pytest.raises(ValueError):
        w.w4a16_gated(x, packed, 64, h=torch.empty((4, 63), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        w.w4a16_gated_grad(x, torch.zeros((4, 64)), packed, 64)  # dh of another type
    with pytest.raises(ValueError):
        w.w4a16_cross_entropy(x, torch.zeros(4, dtype=torch.int64), packed, 1000)
    with pytest.raises(ValueError):
        w.w4a16_cross_entropy(x, torch.zeros(4, dtype=torch.int32), packed, 1000, dloss=torch.ones(4))
    with pytest.raises(ValueError):
        w.w4a16_distill(x, torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 2)), packed, 1000)
