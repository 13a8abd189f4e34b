"""Rows without a target whose logits lie far above their reference (column 0's logit): the
gradient of the others does not leave its usual path for them. The word behind the
workspace's counters (byte 512) says whether it has."""

import pytest
import torch

import train_util as tu
from gpu_util import DEV
from train_util import normal
from test_train_gpu import BF, ULP, logit_eps, rows_within, weight, w  # noqa: F401

pytestmark = pytest.mark.gpu
HOT = 512


def hot(ws):
    return int(ws[HOT:HOT + 4].view(torch.int32)[0])


@pytest.mark.parametrize("M,V", [(20, 1000), (300, 5000), (4096, 40000)])
def test_cross_entropy(w, M, V):  # noqa: F811
    K = 128
    wt = weight(w, K, V, "bf16", 128)
    x, _ = normal(M, (M, K), "bf16")
    x[3::7] = (x[3::7].float() * 60).to(x.dtype)
    lab = torch.arange(M, dtype=torch.int32, device=DEV) % V
    lab[3::7] = -100
    ws = torch.zeros(w.w4a16_cross_entropy_workspace_bytes(M, K, V, 128, True), dtype=torch.uint8, device=DEV)
    out = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True, workspace=ws)
    assert hot(ws) == 0
    x64 = x.double()
    live = (lab >= 0).double()[:, None]
    value, lse, dx, _ = tu.loss(wt.dev64, x64, lab[:, None].long(), live, 1.0, torch.ones(M, dtype=torch.float64, device=DEV))
    eps = logit_eps(x64, K)
    assert ((out[1].double() - lse).abs() <= eps + 2.0 ** -20 * lse.abs()).all()
    assert ((out[0].double() - value).abs() <= 2 * eps + 2.0 ** -20 * (value.abs() + lse.abs())).all()
    rows_within(out[2], dx, 2 * BF + ULP["bf16"], "dx")
    assert (out[2][3::7] == 0).all() and (out[0][3::7] == 0).all()
    # one such row with a target
    lab[3] = 1
    w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True, workspace=ws)
    assert hot(ws) == 1


def test_distill(w):  # noqa: F811
    M, K, V = 70, 128, 3000
    wt = weight(w, K, V, "bf16", 128)
    x, _ = normal(1, (M, K), "bf16")
    x[5], x[6] = (x[5].float() * 60).to(x.dtype), (x[6].float() * 60).to(x.dtype)
    ids = (torch.arange(M * 4, dtype=torch.int32, device=DEV).view(M, 4) * 7) % V
    t = torch.zeros((M, 4), device=DEV)
    ids[5] = -1                                              # no id
    t[6] = -float("inf")                                     # no weight
    ws = torch.zeros(w.w4a16_distill_workspace_bytes(M, K, V, 128, 4, True), dtype=torch.uint8, device=DEV)
    out = w.w4a16_distill(x, ids, t, wt.packed, V, 128, grad=True, workspace=ws)
    assert hot(ws) == 0
    one = torch.ones(M, dtype=torch.float64, device=DEV)
    ref = tu.loss(wt.dev64, x.double(), ids.long(), tu.teacher(ids, t, V, 1.0), 1.0, one)
    eps = logit_eps(x.double(), K)
    assert ((out[1].double() - ref[1]).abs() <= eps + 2.0 ** -20 * ref[1].abs()).all()
    rows_within(out[2], ref[2], 2 * BF + ULP["bf16"], "dx")
    t[6] = 0.0
    w.w4a16_distill(x, ids, t, wt.packed, V, 128, grad=True, workspace=ws)
    assert hot(ws) == 1
