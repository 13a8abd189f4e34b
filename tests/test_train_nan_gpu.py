"""Rows that hold no numbers: their loss and log-sum are no numbers either (0 for the loss
and gradient of a row without a target), and no other row changes."""

import pytest
import torch

from gpu_util import DEV
from train_util import normal
from test_train_gpu import weight, w  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,V,dtype", [(8, 1000, "bf16"), (16, 4104, "fp16"), (24, 1000, "fp16"), (40, 5000, "bf16"),
                                       (300, 2056, "bf16")])
def test_cross_entropy(w, M, V, dtype, grad):  # noqa: F811
    wt = weight(w, 256, V, dtype, 128)
    x, _ = normal(M, (M, 256), dtype)
    lab = torch.arange(M, dtype=torch.int32, device=DEV)
    lab[[2, 5]] = -100
    clean = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=grad)
    dirty = x.clone()
    dirty[1], dirty[2] = float("nan"), float("nan")
    dirty[4], dirty[5] = float("inf"), float("inf")           # every logit is inf - inf
    dirty[7, 3] = float("nan")
    out = w.w4a16_cross_entropy(dirty, lab, wt.packed, V, 128, grad=grad)
    bad = [1, 2, 4, 5, 7]
    assert torch.isnan(out[1][bad]).all()
    assert torch.isnan(out[0][[1, 4, 7]]).all() and (out[0][[2, 5]] == 0).all()
    if grad:
        assert torch.isnan(out[2][[1, 4, 7]].float()).all() and (out[2][[2, 5]] == 0).all()
    keep = [m for m in range(M) if m not in bad]
    for a, b in zip(out, clean):
        assert torch.equal(a[keep].view(torch.uint8), b[keep].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_distill(w, dtype):  # noqa: F811
    M, V = 20, 1000
    wt = weight(w, 256, V, dtype, 128)
    x, _ = normal(3, (M, 256), dtype)
    ids = torch.arange(3 * M, dtype=torch.int32, device=DEV).view(M, 3)
    ids[2] = -1
    t = torch.zeros((M, 3), device=DEV)
    clean = w.w4a16_distill(x, ids, t, wt.packed, V, 128, grad=True)
    dirty = x.clone()
    dirty[1], dirty[2] = float("nan"), float("nan")
    out = w.w4a16_distill(dirty, ids, t, wt.packed, V, 128, grad=True)
    assert torch.isnan(out[1][[1, 2]]).all() and torch.isnan(out[0][1]) and out[0][2] == 0
    assert torch.isnan(out[2][1].float()).all() and (out[2][2] == 0).all()
    keep = [m for m in range(M) if m not in (1, 2)]
    for a, b in zip(out, clean):
        assert torch.equal(a[keep].view(torch.uint8), b[keep].view(torch.uint8))
