"""The differentiable operations' own logic, on functions that stand in for the library's."""

import pytest
import torch

from w4a16_int4_weight_amd import autograd as ops

K, V = 128, 64


class Losses:
    """Stand-ins whose gradient is dloss[m] * base, rounded to x's type."""

    def __init__(self, monkeypatch):
        self.asked = []
        monkeypatch.setattr(ops, "w4a16_cross_entropy", self.cross_entropy)
        monkeypatch.setattr(ops, "w4a16_distill", self.distill)

    def base(self, x):
        return x.float() * 0.25 + 0.5

    def cross_entropy(self, x, labels, packed, V, group_size, dloss=None, grad=False):
        self.asked.append(grad)
        M = x.shape[0]
        out = (torch.arange(M, dtype=torch.float32), torch.zeros(M))
        if not grad:
            assert dloss is None
            return out
        d = torch.ones(M) if dloss is None else dloss
        return (*out, (d[:, None] * self.base(x)).to(x.dtype))

    def distill(self, x, ids, top, packed, V, group_size, temperature=1.0, dloss=None, grad=False):
        return self.cross_entropy(x, ids, packed, V, group_size, dloss, grad)


@pytest.fixture
def losses(monkeypatch):
    return Losses(monkeypatch)


def both(x, weights=None, top=None):
    """-> the two losses' calls on x [M, K]"""
    M = x.shape[0]
    labels, ids = torch.zeros(M, dtype=torch.int32), torch.zeros((M, 3), dtype=torch.int32)
    top = torch.zeros((M, 3)) if top is None else top
    return [lambda: ops.cross_entropy(x, labels, None, V, weights=weights),
            lambda: ops.distill(x, ids, top, None, V, weights=weights)]


@pytest.mark.parametrize("i", [0, 1])
def test_no_gradient_where_none_is_asked_for(losses, i):
    x = torch.randn((4, K)).to(torch.bfloat16).requires_grad_(True)
    weights = torch.full((4,), 0.25)
    with torch.no_grad():
        assert not both(x, weights)[i]().requires_grad
    with torch.inference_mode():
        both(x, weights)[i]()
    both(x.detach(), weights)[i]()
    assert losses.asked == [False, False, False]
    # a checkpoint's first pass forms none, its second does
    from torch.utils.checkpoint import checkpoint
    checkpoint(lambda v: both(v, weights)[i](), x, use_reentrant=True).sum().backward()
    assert losses.asked[3:] == [False, True]
    assert torch.equal(x.grad, (0.25 * losses.base(x)).to(x.dtype))


@pytest.mark.parametrize("need", [False, True])
def test_constants_that_require_a_gradient_are_refused(losses, monkeypatch, need):
    monkeypatch.setattr(ops, "w4a16_gemm", lambda x, packed, N, group_size, bias=None: torch.zeros((x.shape[0], N)))
    x = torch.randn((4, K)).to(torch.bfloat16).requires_grad_(need)
    weights, top = torch.ones(4, requires_grad=True), torch.zeros((4, 3), requires_grad=True)
    bias = torch.zeros(V, requires_grad=True)
    calls = [both(x, weights)[0], both(x, weights)[1], both(x, top=top)[1],
             lambda: ops.linear(x, torch.zeros(1, dtype=torch.uint8), V, bias=bias)]
    for call in calls:
        with pytest.raises(ValueError, match="detach"):
            call()
        with torch.no_grad():
            call()
    for call in both(x, weights.detach(), top.detach()):
        call()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 65536.0])
@pytest.mark.parametrize("weight", [2.0 ** -13, 1e-7, 1.0 / 24576, 0.0, 0.75])
def test_a_scale_on_the_loss_reaches_small_gradients(losses, dtype, scale, weight):
    # one rounding of weight * base, relative: half a step of the type; where the result with
    # the scale is below the type's normal range, half a step there
    x = torch.randn((6, K)).clamp(-1, 1).to(dtype).requires_grad_(True)
    weights = torch.full((6,), weight)
    info = torch.finfo(dtype)
    for i in (0, 1):
        x.grad = None
        (both(x, weights)[i]().sum() * scale).backward()
        want = losses.base(x.detach()).double() * float(weights[0]) * scale
        err = (x.grad.double() - want).abs()
        assert (err <= info.eps / 2 * want.abs() * 1.001 + info.tiny * info.eps / 2 * 1.001).all()


def test_linear_refuses_what_is_elsewhere(monkeypatch):
    monkeypatch.setattr(ops, "w4a16_gemm", lambda *args, **more: pytest.fail("called"))
    x, packed = torch.zeros((4, K), dtype=torch.bfloat16), torch.zeros(1 << 15, dtype=torch.uint8)
    with pytest.raises(ValueError, match="bias"):
        ops.linear(x, packed, V, bias=torch.zeros(V, dtype=torch.bfloat16, device="meta"))
    with pytest.raises(ValueError, match="packed"):
        ops.linear(x, packed.to("meta"), V)
