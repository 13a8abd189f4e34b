"""The differentiable operations and the example that runs them together."""

import os
import sys

import pytest
import torch

import train_util as tu
from gpu_util import DEV
from train_util import normal
from test_train_gpu import BF, ULP, rows_within, weight, w  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gradients(w, dtype):  # noqa: F811
    from w4a16_int4_weight_amd import autograd as ops
    K, F, V, G = 256, 264, 1000, 64
    up, down, head = weight(w, K, 2 * F, dtype, G), weight(w, 128, K, dtype, -1), weight(w, K, V, dtype, G)
    x, x64 = normal(1, (3, 7, K), dtype)
    # gated
    xg = x.clone().requires_grad_(True)
    h = ops.gated(xg, up.packed, F, G, act="gelu")
    assert h.shape == (3, 7, F)
    dh, dh64 = normal(2, (3, 7, F), dtype)
    h.backward(dh)
    ref = tu.gated_grad(up.dev64, F, x64.view(21, K), dh64.view(21, F), "gelu")
    rows_within(xg.grad.view(21, K), ref, 2 * BF + ULP[dtype], "gated")
    # linear, from a gradient that is a view with strides
    xl = normal(3, (21, 128), dtype)[0].requires_grad_(True)
    y = ops.linear(xl, down.packed, K, -1)
    dy, dy64 = normal(4, (K, 21), dtype)
    y.backward(dy.t())
    rows_within(xl.grad, dy64.t() @ down.dev64.t(), 2 * ULP[dtype], "linear")
    # losses: the weighted sum, its gradient, rows without a target
    lab = torch.arange(21, dtype=torch.int32, device=DEV).view(3, 7) * 40
    lab[1, 2] = -100
    weights = torch.linspace(0.5, 2.0, 21, device=DEV).view(3, 7)
    xc = x.clone().requires_grad_(True)
    loss = ops.cross_entropy(xc, lab, head.packed, V, G, weights=weights)
    loss.sum().backward()
    flat, wd = lab.view(-1, 1).long(), weights.view(-1).double()
    value, _, dx, _ = tu.loss(head.dev64, x64.view(21, K), flat, ((flat >= 0) & (flat < V)).double(), 1.0, wd)
    assert loss.shape == lab.shape and torch.allclose(loss.detach().view(-1).double(), value * wd, rtol=2 ** -16, atol=2 ** -16)
    rows_within(xc.grad.view(21, K), dx, 2 * BF + ULP[dtype], "cross entropy")
    assert (xc.grad[1, 2] == 0).all()
    ids = torch.randperm(V, device=DEV)[:21 * 6].view(3, 7, 6).to(torch.int32)
    t = torch.randn((3, 7, 6), device=DEV)
    xd = x.clone().requires_grad_(True)
    ops.distill(xd, ids, t, head.packed, V, G, temperature=2.0).sum().backward()
    p = tu.teacher(ids.view(21, 6), t.view(21, 6), V, 2.0)
    dx = tu.loss(head.dev64, x64.view(21, K), ids.view(21, 6).long(), p, 2.0, torch.ones(21, dtype=torch.float64, device=DEV))[2]
    rows_within(xd.grad.view(21, K), dx, 2 * BF + ULP[dtype], "distill")
    with torch.no_grad():                                  # no gradient asked for: none formed
        assert not ops.cross_entropy(x, lab, head.packed, V, G).requires_grad


def test_training_step_in_a_graph(w):  # noqa: F811
    # forward and backward captured once, replayed on other inputs between eager work
    from w4a16_int4_weight_amd import autograd as ops
    K, F, V, M = 256, 256, 1000, 32
    up, head = weight(w, K, 2 * F, "bf16", 128), weight(w, F, V, "bf16", 128)
    lab = torch.arange(M, dtype=torch.int32, device=DEV) * 11
    xs = [normal(60 + i, (M, K), "bf16")[0] for i in range(3)]

    def step(x):
        leaf = x.detach().requires_grad_(True)
        loss = ops.cross_entropy(ops.gated(leaf, up.packed, F), lab, head.packed, V).sum()
        return loss.detach(), torch.autograd.grad(loss, leaf)[0]

    want = [step(x) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss, dx = step(x)
    for i in (0, 1, 2, 1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want[i][1]) and torch.allclose(loss, want[i][0], rtol=2 ** -20)
        step(xs[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_example_learns(dtype):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import adapt_int4
    ce, kd, scores = adapt_int4.run(steps=15, dtype=dtype)
    assert ce[-1] < ce[0] - 0.5 and kd[-1] < kd[0]
    assert torch.isfinite(scores).all() and (scores < 0).all()
