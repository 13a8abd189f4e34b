"""Rows that are sure of their target: the loss and the gradient are small, and still right
relative to themselves. With w = sum_{v != t} e^{z_v - z_t}, the loss is log(1 + w): an error
of 2 eps in a difference of logits (logit_eps) is one of 2 eps in w, and exp and the sum add
2^-20. The gradient's roundings are P's, W's and dx's to the type, and the target's share is
off by w's error too."""

import pytest
import torch

import train_util as tu
from gpu_util import DEV, TORCH_DTYPE
from train_util import ULP
from test_train_gpu import logit_eps, rows_within, weight, w  # noqa: F401

pytestmark = pytest.mark.gpu


def rows(wt, M, V, dtype):
    """x along the labels' columns (and a little of everything), as sure as the row's number says"""
    gen = torch.Generator(device=DEV).manual_seed(M)
    lab = torch.randint(0, V, (M,), generator=gen, device=DEV)
    lab[0], lab[-1] = V - 1, 0
    along = wt.dev64[:, lab].t()
    noise = torch.randn((M, wt.K), generator=gen, device=DEV, dtype=torch.float64)
    x = (along / along.norm(dim=1, keepdim=True) * torch.linspace(2.0, 30.0, M, device=DEV)[:, None].double()
         + 0.1 * noise).to(TORCH_DTYPE[dtype]).contiguous()
    z = x.double() @ wt.dev64
    zt = z.gather(1, lab[:, None])
    odds = torch.exp(z - zt).scatter(1, lab[:, None], 0.0).sum(1)
    return x, lab.to(torch.int32), z, zt[:, 0], odds


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,V", [(5, 512, 2000), (16, 1024, 5000), (40, 512, 2000), (300, 384, 1032)])
def test_cross_entropy(w, M, K, V, dtype):  # noqa: F811
    wt = weight(w, K, V, dtype, 128)
    x, lab, z, zt, odds = rows(wt, M, V, dtype)
    assert float(odds.min()) < 1e-4
    loss64 = torch.log1p(odds)
    eps = 2 * logit_eps(x.double(), K) + 2.0 ** -20
    grad = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True, dloss=(1 / -torch.expm1(-loss64)).float())
    for out in (w.w4a16_cross_entropy(x, lab, wt.packed, V, 128), grad):
        assert (out[0] >= 0).all()
        assert ((out[0].double() - loss64).abs() <= 1.5 * eps * loss64 + 1e-37).all()     # (1.5: the log's own slope)
        assert ((out[1].double() - zt - loss64).abs() <= eps + 2.0 ** -20 * out[1].abs()).all()
    # dloss = 1 / (1 - q_t): the gradient is of order one in every row
    q = torch.exp(z - (zt + loss64)[:, None]).scatter(1, lab[:, None].long(), 0.0)
    dx = (q @ wt.dev64.t() + torch.expm1(-loss64)[:, None] * wt.dev64[:, lab.long()].t()) / -torch.expm1(-loss64)[:, None]
    rows_within(grad[2], dx, 3 * ULP[dtype] + 4 * float(eps.max()), "dx")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_distillation_from_one_entry(w, dtype):  # noqa: F811
    M, K, V = 30, 512, 2000
    wt = weight(w, K, V, dtype, 128)
    x, lab, z, zt, odds = rows(wt, M, V, dtype)
    ids, t = lab[:, None].contiguous(), torch.zeros((M, 1), device=DEV)
    t[4], ids[5] = -float("inf"), -1                                    # nothing left
    t[6] = float("nan")
    dloss = (1 / -torch.expm1(-torch.log1p(odds))).float()
    ce = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True, dloss=dloss)
    di = w.w4a16_distill(x, ids, t, wt.packed, V, 128, grad=True, dloss=dloss)
    assert (di[0][[4, 5]] == 0).all() and (di[2][[4, 5]] == 0).all()
    lse = torch.logsumexp(z, 1)
    assert ((di[1].double() - lse).abs() <= 2 * logit_eps(x.double(), K) + 2.0 ** -20 * lse.abs()).all()
    assert torch.isnan(di[0][6]) and torch.isnan(di[2][6].float()).all()
    keep = [m for m in range(M) if m not in (4, 5, 6)]
    for a, b in zip(ce, di):
        assert torch.equal(a[keep], b[keep])
