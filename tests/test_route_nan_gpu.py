"""The router's rows in which some score is no number: T different experts, and weights that are none."""

import pytest
import torch

import serve_util as su
from gpu_util import DEV, TORCH_DTYPE

pytestmark = pytest.mark.gpu

T = 5
MODES = [(score, normalize, bias) for score in ("softmax", "sigmoid") for normalize in (True, False) for bias in (True, False)]
# a wave an expert, and tiles of 16 rows x 16 experts; 1, 2, 4 and 16 experts a lane
SIZES = [(4, 12), (4, 80), (130, 12), (40, 200), (130, 80), (20, 1000)]


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


def make(M, E, dtype="bf16", K=256):
    gen = torch.Generator().manual_seed(31 * M + E)
    x = torch.randn((M, K), generator=gen).to(TORCH_DTYPE[dtype]).to(DEV)
    router = (torch.randn((E, K), generator=gen) * 1.5 / K ** 0.5).to(TORCH_DTYPE[dtype]).to(DEV)
    return x, router, (torch.randn((E,), generator=gen) * 0.1).to(DEV)


def different(ids, E):
    ids = ids.long().cpu()
    return all(len(set(r)) == T and min(r) >= 0 and max(r) < E for r in ids.tolist())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,E", SIZES)
def test_one_expert_of_no_numbers(w, M, E, dtype):
    """One row of the router is broken: one l of every row is no number, wherever the expert stands."""
    x, router, bias = make(M, E, dtype)
    for bad in (0, E // 2, E - 1):
        broken = router.clone()
        broken[bad, 17] = float("nan")
        for score, normalize, biased in MODES:
            ids, weights = w.w4a16_route(x, broken, T, bias=bias if biased else None, score=score, normalize=normalize, scale=2.0)
            assert different(ids, E), (bad, score, normalize, biased)
            assert bool(torch.isnan(weights).all()), (bad, score, normalize, biased)


@pytest.mark.parametrize("M,E", SIZES)
def test_other_rows_are_what_they_are(w, M, E):
    """A row of x with an entry that is no number: its weights are none, the others' are the definition's."""
    x, router, bias = make(M, E)
    x[2, 9] = float("nan")
    rest = [m for m in range(M) if m != 2]
    for score, normalize, biased in MODES:
        how = dict(bias=bias if biased else None, score=score, normalize=normalize)
        ids, weights = w.w4a16_route(x, router, T, **how)
        assert different(ids, E) and bool(torch.isnan(weights[2]).all())
        want, ww = su.route(x[rest].double(), router.double(), T, **how)
        assert torch.equal(ids[rest].long(), want)
        assert ((weights[rest].double() - ww).abs() <= 2.0 ** -24 * ww.abs() * 1.001 + 1e-38).all()


@pytest.mark.parametrize("M,E", SIZES)
def test_infinite_products(w, M, E):
    """An expert whose l is infinite: under softmax +infinity leaves a row no weights, -infinity is a weight of 0;
    a sigmoid is 1 or 0."""
    x, router, bias = make(M, E)
    router[E // 3, 5] = float("inf")
    for score, normalize, biased in MODES:
        how = dict(bias=bias if biased else None, score=score, normalize=normalize)
        ids, weights = w.w4a16_route(x, router, T, **how)
        assert different(ids, E)
        want, ww = su.route(x.double(), router.double(), T, **how)
        lost = (x[:, 5] > 0) & (score == "softmax")
        assert bool(lost.any()) == (score == "softmax") and not bool(lost.all())
        assert bool(torch.isnan(weights[lost]).all())
        assert torch.equal(ids[~lost].long(), want[~lost])
        assert ((weights[~lost].double() - ww[~lost]).abs() <= 2.0 ** -24 * ww[~lost].abs() * 1.001 + 1e-38).all()


@pytest.mark.parametrize("M", [4, 40])
def test_the_layer_hides_nothing(w, M):
    ex = su.Experts(w, 900, 6, 256, 128, "bf16", 128)
    x, router, _ = make(M, 6)
    router[3, 0] = float("nan")
    y, ids, weights = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, 128, T, 128)
    assert different(ids, 6) and bool(torch.isnan(weights).all()) and bool(torch.isnan(y.float()).all())
