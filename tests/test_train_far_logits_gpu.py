"""Losses whose logits lie far from the row's reference (its largest target logit): the
tiles that hold them take references of their own, over several tiles and pieces of the
vocabulary. Tolerances as in test_train_gpu, and one rounding more for a tile's factor."""

import numpy as np
import pytest
import torch

import train_util as tu
from gpu_util import DEV
from train_util import normal
from test_train_gpu import BF, ULP, logit_eps, rows_within, weight, w  # noqa: F401

pytestmark = pytest.mark.gpu


def check(w, M, K, V, dtype, scale, seed, tau=1.0):  # noqa: F811
    print(f"far logits M={M} K={K} V={V} {dtype} scale={scale}", flush=True)
    wt = weight(w, K, V, dtype, 128)
    x, _ = normal(seed, (M, K), dtype)
    x = (x.float() * scale[:M, None]).to(x.dtype)
    x64 = x.double()
    lab = torch.from_numpy(np.random.default_rng(seed).integers(0, V, M).astype(np.int32)).to(DEV)
    lab[::7] = -100                                       # their reference is column 0's logit
    out = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True)
    torch.cuda.synchronize()
    p = (lab >= 0).double()[:, None]
    value, lse, dx, _ = tu.loss(wt.dev64, x64, lab[:, None].long(), p, 1.0, torch.ones(M, dtype=torch.float64, device=DEV))
    eps = logit_eps(x64, K)
    assert ((out[1].double() - lse).abs() <= eps + 2.0 ** -20 * lse.abs()).all()
    assert ((out[0].double() - value).abs() <= 2 * eps + 2.0 ** -20 * (value.abs() + lse.abs())).all()
    # q is off by its logit's and the log-sum's error; a row's gradient is at least 2^-24
    # of what it is a difference of
    rows_within(out[2], dx + 0.0, 3 * BF + ULP[dtype] + 4 * float(eps.max()), "dx")
    plain = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128)
    assert ((plain[1].double() - lse).abs() <= eps + 2.0 ** -20 * lse.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,V", [(1, 3000), (40, 3000), (300, 2056)])
def test_every_row_far(w, M, V, dtype):  # noqa: F811
    check(w, M, 256, V, dtype, torch.full((M,), 60.0, device=DEV), 40 + M)


def test_some_rows_far_over_pieces(w):  # noqa: F811
    # two pieces: rows as usual, far ones whose maximum is in either piece
    M, V = 4096, 33000
    scale = torch.ones(M, device=DEV)
    scale[5::64] = 80.0
    scale[6::64] = 300.0
    check(w, M, 128, V, "bf16", scale, 77)


def test_distill_far(w):  # noqa: F811
    M, K, V, T = 50, 256, 3000, 16
    wt = weight(w, K, V, "bf16", 128)
    x, x64 = normal(3, (M, K), "bf16", scale=50.0)
    rng = np.random.default_rng(8)
    ids = torch.from_numpy(np.stack([rng.choice(V, T, replace=False) for _ in range(M)]).astype(np.int32)).to(DEV)
    t = torch.from_numpy((3 * rng.standard_normal((M, T))).astype(np.float32)).to(DEV)
    out = w.w4a16_distill(x, ids, t, wt.packed, V, 128, temperature=2.0, grad=True)
    ref = tu.loss(wt.dev64, x64, ids.long(), tu.teacher(ids, t, V, 2.0), 2.0, torch.ones(M, dtype=torch.float64, device=DEV))
    eps = logit_eps(x64, K) / 2
    assert ((out[0].double() - ref[0]).abs() <= 4 * 2 * eps + 2.0 ** -20 * (ref[0].abs() + 4 * ref[1].abs())).all()
    rows_within(out[2], ref[2], 3 * BF + ULP["bf16"] + 4 * float(eps.max()), "dx")
