"""Every instantiation of the training and scoring kernels against 64 bits: all tile heights,
group sizes, types, splits of K and of the sum over columns (train_plans.py says which shape
takes which, and a CPU test that none is left out), and each against itself.

Tolerances count roundings, each at most half a step (ULP: bf16 2^-8, fp16 2^-11, relative),
which in the norm of a row add up to less than their sum:
  dx = dy W^T    W and dx, to the type
  gated          h, and the fp32 errors of g and u (test_train_gpu's)
  its backward   dx to the type; dg | du and W to fp16. Where fp16 keeps what dg | du's
                 rounding leaves (tiles of up to 128 rows) theirs is 2^-21
  losses         P, W and dx to the type
and twice (four times, for a q that is off by its logit's and the log-sum's) the largest fp32
error of a logit, logit_eps, which meets values of order one. A row whose gradient is tiny
meets two limits that are no kernel's: fp16's step below its normal range (2^-24, half of it
for each element), and the 64-bit reference's own softmax less one (2^-50 of the column)."""

import pytest
import torch

import train_plans as tp
import train_util as tu
from gpu_util import DEV, TORCH_DTYPE
from train_util import ULP, normal
from test_train_gpu import check_loss, logit_eps, rows_within, w  # noqa: F401

pytestmark = pytest.mark.gpu
FP16 = 2.0 ** -11
_kept = {}


class Weight:
    """Random checkpoint tensors (codes along K), packed, and their values in 64 bits."""

    def __init__(self, w, K, N, dtype, G):  # noqa: F811
        gen = torch.Generator(device=DEV).manual_seed(K + N + G)
        word = lambda *shape: torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen, device=DEV).to(torch.int32)  # noqa: E731
        qweight, qzeros = word(K // 8, N), word(K // G, N // 8)
        scales = (torch.rand((K // G, N), generator=gen, device=DEV) * 0.015 + 0.005).to(TORCH_DTYPE[dtype])
        self.packed = w.w4a16_repack_gptq(qweight, qzeros, scales, G)
        nibble = 4 * torch.arange(8, dtype=torch.int32, device=DEV)
        q = ((qweight[:, None, :] >> nibble[None, :, None]) & 15).view(K // G, G, N)
        z = ((qzeros[:, :, None] >> nibble[None, None, :]) & 15).view(K // G, 1, N)
        self.W = ((q - z).double() * scales.double()[:, None, :]).view(K, N)


def weight(w, K, N, dtype, G):  # noqa: F811
    key = (K, N, dtype, G)
    if key not in _kept:
        _kept.clear()
        _kept[key] = Weight(w, K, N, dtype, G)
    return _kept[key]


def check(out, ref, W, x64, K, lab, dtype, tol):  # noqa: F811
    """check_loss with those two limits for the gradient"""
    check_loss(out[:2], ref, x64, K, 1.0, dtype, tol)
    if len(out) == 3:
        assert torch.isfinite(out[2].float()).all()
        err, size = (out[2].double() - ref[2]).norm(dim=1), ref[2].norm(dim=1)
        column = W.norm(dim=0)[lab.clamp(min=0).long()]
        lim = tol * size + (2.0 ** -25 * K ** 0.5 if dtype == "fp16" else 0.0) + 2.0 ** -50 * column
        bad = (err > lim).nonzero().flatten()
        assert bad.numel() == 0, f"rows {bad[:8].tolist()}, worst {float((err / lim).max()):.2f} of the tolerance"


def same(a, b):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


every = [pytest.mark.parametrize("G", tp.GROUPS), pytest.mark.parametrize("dtype", tp.DTYPES)]


def cases(shapes):
    def mark(f):
        for m in every:
            f = m(f)
        return pytest.mark.parametrize("M,K,N", shapes)(f)
    return mark


@cases(tp.GEMM_GRAD)
def test_gemm_grad(w, M, K, N, dtype, G):  # noqa: F811
    wt = weight(w, K, N, dtype, G)
    dy, dy64 = normal(M + N, (M, N), dtype)
    dx = w.w4a16_gemm_grad(dy, wt.packed, K, G)
    rows_within(dx, dy64 @ wt.W.t(), 2 * ULP[dtype], "dx")
    same(dx, w.w4a16_gemm_grad(dy, wt.packed, K, G))


@cases(tp.GATED)
def test_gated(w, M, K, N, dtype, G):  # noqa: F811
    act = ["silu", "gelu", "gelu_tanh"][(M + G // 32) % 3]
    wt = weight(w, K, 2 * N, dtype, G)
    x, x64 = normal(M + N, (M, K), dtype)
    g, u = x64 @ wt.W[:, :N], x64 @ wt.W[:, N:]
    eps = logit_eps(x64, K)
    h = w.w4a16_gated(x, wt.packed, N, G, act=act)
    a = tu.act(act, g)
    slack = eps[:, None] * (1.13 * u.abs() + a.abs()) + 2.0 ** -20 * (g * u).abs()
    worst = ((h.double() - a * u).abs() / (ULP[dtype] * (a * u).abs() + slack + 2.0 ** -25)).max()
    assert float(worst) <= 1.0, float(worst)
    same(h, w.w4a16_gated(x, wt.packed, N, G, act=act))

    dh, dh64 = normal(M + 1, (M, N), dtype)
    dx = w.w4a16_gated_grad(x, dh, wt.packed, N, G, act=act)
    rest = dtype == "fp16" and tp.grad(w, M, K, 2 * N).bm <= 128
    inner = 2.0 ** -21 if rest else FP16
    rows_within(dx, tu.gated_grad(wt.W, N, x64, dh64, act), ULP[dtype] + FP16 + inner + 2 * float(eps.max()), "dx")
    same(dx, w.w4a16_gated_grad(x, dh, wt.packed, N, G, act=act))


@cases(tp.LOSS)
def test_cross_entropy(w, M, K, N, dtype, G):  # noqa: F811
    wt = weight(w, K, N, dtype, G)
    x, x64 = normal(M + N, (M, K), dtype)
    lab = torch.randint(0, N, (M,), generator=torch.Generator(device=DEV).manual_seed(M), device=DEV).to(torch.int32)
    lab[3::9] = -100
    dloss = torch.linspace(0.5, 2.0, M, device=DEV)
    ref = tu.loss(wt.W, x64, lab[:, None].long(), (lab >= 0).double()[:, None], 1.0, dloss.double())
    tol = 3 * ULP[dtype] + 4 * float(logit_eps(x64, K).max())
    out = w.w4a16_cross_entropy(x, lab, wt.packed, N, G)
    check(out, ref, wt.W, x64, K, lab, dtype, tol)
    full = w.w4a16_cross_entropy(x, lab, wt.packed, N, G, grad=True, dloss=dloss)
    check(full, ref, wt.W, x64, K, lab, dtype, tol)
    for a, b in zip(full, w.w4a16_cross_entropy(x, lab, wt.packed, N, G, grad=True, dloss=dloss)):
        same(a, b)


@pytest.mark.parametrize("G", [128, 32])
@pytest.mark.parametrize("M,K,N", [s for s in tp.LOSS if s[2] < 10000])
def test_cross_entropy_far(w, M, K, N, G):  # noqa: F811
    # rows whose logits lie far from their reference: the tiles' own references, and the
    # product with W^T that rescales them (bf16), one rounding more
    wt = weight(w, K, N, "bf16", G)
    x, _ = normal(M + 2, (M, K), "bf16")
    x[::5] = (x[::5].float() * 24).to(x.dtype)
    x64 = x.double()
    lab = torch.randint(0, N, (M,), generator=torch.Generator(device=DEV).manual_seed(M), device=DEV).to(torch.int32)
    one = torch.ones(M, dtype=torch.float64, device=DEV)
    ref = tu.loss(wt.W, x64, lab[:, None].long(), one[:, None], 1.0, one)
    out = w.w4a16_cross_entropy(x, lab, wt.packed, N, G, grad=True)
    check(out, ref, wt.W, x64, K, lab, "bf16", 4 * ULP["bf16"] + 4 * float(logit_eps(x64, K).max()))
