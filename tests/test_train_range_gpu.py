"""The gated block's backward at the ends of fp32's range: dg and du that only a power of
two brings into fp16, and whose product is still finite.

Tolerances: dx is rounded once to its type, dg | du and the weights once each to fp16 (2^-11
relative at most), in the norm no more than their sum."""

import pytest
import torch

import train_util as tu
from gpu_util import DEV
from train_util import ULP, normal
from test_train_gpu import rows_within, weight, w  # noqa: F401

pytestmark = pytest.mark.gpu
FP16 = 2.0 ** -11


@pytest.mark.parametrize("scale", [1e37, 1e36, 1e34, 1e30, 1e-30, 1e-35, 1e-36])
@pytest.mark.parametrize("M,F", [(4, 40), (4, 264), (40, 40), (40, 264), (150, 1000)])
def test_gated_grad_far_scales(w, M, F, scale):  # noqa: F811
    K = 256
    wt = weight(w, K, 2 * F, "bf16", 128)
    x, x64 = normal(M, (M, K), "bf16", scale=0.3)
    dh = (normal(M + F, (M, F), "bf16")[0].float().clamp(-2, 2) * scale).to(torch.bfloat16)
    # rows of several scales: each has its own
    dh[1::3] = (dh[1::3].float() * 2.0 ** (-60 if scale > 1 else 60)).to(torch.bfloat16)
    ref = tu.gated_grad(wt.dev64, F, x64, dh.double(), "silu")
    assert float(ref.abs().max()) < 1e38
    dx = w.w4a16_gated_grad(x, dh, wt.packed, F, 128)
    rows_within(dx.double() / scale, ref / scale, ULP["bf16"] + 2 * FP16, "dx")


def test_infinite_gradients_stay_in_their_rows(w):  # noqa: F811
    M, K, F = 40, 256, 264
    wt = weight(w, K, 2 * F, "bf16", 128)
    x, _ = normal(5, (M, K), "bf16")
    dh, _ = normal(6, (M, F), "bf16")
    clean = w.w4a16_gated_grad(x, dh, wt.packed, F, 128)
    dh[3, 5], dh[9, 7] = float("inf"), float("nan")
    dx = w.w4a16_gated_grad(x, dh, wt.packed, F, 128)
    keep = torch.tensor([m for m in range(M) if m not in (3, 9)], device=DEV)
    assert torch.equal(dx[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert torch.isnan(dx[9].float()).all() and not torch.isfinite(dx[3].float()).any()
