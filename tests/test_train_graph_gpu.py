"""Captured training steps with no workspace passed: replays among eager calls that need
larger workspaces on the capture's stream, and graphs captured on a stream that has had none."""

import pytest
import torch

from gpu_util import DEV
from train_util import normal
from test_train_gpu import weight, w  # noqa: F401

pytestmark = pytest.mark.gpu


def steps(w, M, seed):  # noqa: F811
    """-> (step(x): loss, lse, gradients through every multi-launch entry), three inputs"""
    K, F, V = 256, 512, 2000
    up, down, head = (weight(w, K, n, "bf16", 128).packed for n in (2 * F, F, V))
    lab = torch.arange(M, dtype=torch.int32, device=DEV) % V
    ids = (lab[:, None] + 7 * torch.arange(5, dtype=torch.int32, device=DEV)[None, :]) % V
    ids, top = ids.to(torch.int32).contiguous(), torch.zeros((M, 5), device=DEV)

    def step(x):
        ce = w.w4a16_cross_entropy(x, lab, head, V, grad=True)
        kd = w.w4a16_distill(x, ids, top, head, V, grad=True)
        h = w.w4a16_gated(x, up, F)
        return (*ce, *kd, h, w.w4a16_gated_grad(x, h, up, F), w.w4a16_gemm_grad(h, down, K))
    return step, [normal(seed + i, (M, K), "bf16")[0] for i in range(3)]


def same(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def capture(step, x, stream):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = step(x)
    torch.cuda.synchronize()
    return graph, out


def test_replay_after_a_larger_eager_call(w):  # noqa: F811
    step, xs = steps(w, 40, 100)
    large, big = steps(w, 700, 200)
    want, want_large = [step(x) for x in xs], large(big[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        same(step(xs[0]), want[0])                        # a warm-up with the workspace it needs
    x = xs[0].clone()
    graph, out = capture(step, x, side)
    with torch.cuda.stream(side):
        same(large(big[0]), want_large)                   # the stream's own workspace is replaced
        others = [torch.full((1 << 20,), 3, dtype=torch.uint8, device=DEV) for _ in range(64)]
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        same(out, want[i])
        with torch.cuda.stream(side):
            same(step(xs[2]), want[2])
        torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in others)


def test_first_use_of_a_stream_in_captures(w):  # noqa: F811
    # no eager call before: each graph brings and clears its own workspace, and the second is
    # replayed before the first, after eager calls on the stream
    step, xs = steps(w, 40, 300)
    want = [step(x) for x in xs]
    side = torch.cuda.Stream()
    x = xs[0].clone()
    first, out1 = capture(step, x, side)
    second, out2 = capture(step, x, side)
    with torch.cuda.stream(side):
        same(step(xs[1]), want[1])
    torch.cuda.synchronize()
    for graph, out, i in ((second, out2, 1), (first, out1, 2), (second, out2, 0), (second, out2, 2), (first, out1, 1)):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        same(out, want[i])
        same(step(xs[0]), want[0])


def test_split_product_in_a_capture(w):  # noqa: F811
    # the one-launch entries share the workspace, and its counters, with the others
    K, V, M = 6656, 512, 16
    wt = weight(w, K, V, "bf16", 128)
    xs = [normal(400 + i, (M, K), "bf16")[0] for i in range(2)]
    assert w.w4a16_workspace_bytes(M, K, V, 128) > 0

    def step(x):
        y = w.w4a16_gemm(x, wt.packed, V, 128)
        return y, w.w4a16_gemm_grad(y, wt.packed, K, 128), w.w4a16_gemm(x, wt.packed, V, 128)
    want = [step(x) for x in xs]
    x = xs[0].clone()
    graph, out = capture(step, x, torch.cuda.Stream())
    for i in (0, 1, 1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        same(out, want[i])
        same(step(xs[1 - i]), want[1 - i])
