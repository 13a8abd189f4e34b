"""fp16 losses under a loss scale: the gradients that 1 / count makes too small for fp16 come
back whole. Roundings of fp16, at most 2^-11 relative each: P, W and dx, and one more where
the factor on the loss is no power of two."""

import pytest
import torch

import train_util as tu
from gpu_util import DEV
from train_util import ULP, normal
from test_train_gpu import rows_within, weight, w  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale,roundings", [(65536.0, 3), (40000.0, 4)])
@pytest.mark.parametrize("M,V", [(10, 1000), (333, 5000)])
def test_small_weights(w, M, V, scale, roundings):  # noqa: F811
    from w4a16_int4_weight_amd import autograd as ops
    K = 256
    wt = weight(w, K, V, "fp16", 128)
    x, x64 = normal(M, (M, K), "fp16")
    weights = torch.linspace(0.2, 1.0, M, device=DEV) / 8192
    weights[4] = 0.0
    lab = torch.arange(M, dtype=torch.int32, device=DEV) * 2
    ids = (lab[:, None] + torch.arange(4, dtype=torch.int32, device=DEV)[None, :] * 3).to(torch.int32).contiguous()
    top = torch.randn((M, 4), device=DEV)
    factor = weights.double() * scale

    leaf = x.clone().requires_grad_(True)
    loss = ops.cross_entropy(leaf, lab, wt.packed, V, weights=weights)
    (loss.sum() * scale).backward()
    value, _, dx, _ = tu.loss(wt.dev64, x64, lab[:, None].long(), torch.ones((M, 1), dtype=torch.float64, device=DEV), 1.0, factor)
    assert torch.allclose(loss.detach().double() * scale, value * factor, rtol=2 ** -16, atol=2 ** -16)
    rows_within(leaf.grad, dx, roundings * ULP["fp16"], "cross entropy")

    leaf = x.clone().requires_grad_(True)
    (ops.distill(leaf, ids, top, wt.packed, V, temperature=2.0, weights=weights).sum() * scale).backward()
    dx = tu.loss(wt.dev64, x64, ids.long(), tu.teacher(ids, top, V, 2.0), 2.0, factor)[2]
    rows_within(leaf.grad, dx, roundings * ULP["fp16"], "distill")
