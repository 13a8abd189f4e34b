"""The router against its definition in 64 bits."""

import pytest
import torch

import serve_util as su
from gpu_util import DEV, TORCH_DTYPE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


def make(seed, M, K, E, dtype):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=gen).to(TORCH_DTYPE[dtype]).to(DEV)
    router = (torch.randn((E, K), generator=gen) * 1.5 / K ** 0.5).to(TORCH_DTYPE[dtype]).to(DEV)
    bias = (torch.randn((E,), generator=gen) * 0.1).to(DEV)
    return x, router, bias


def check(w, x, router, T, **how):
    ids, weights = w.w4a16_route(x, router, T, **how)
    want, ww = su.route(x.double(), router.double(), T, **how)
    assert torch.equal(ids.long(), want)
    # one rounding to fp32 (half a step: 2^-24), the rest in fp64
    assert ((weights.double() - ww).abs() <= 2.0 ** -24 * ww.abs() * 1.001 + 1e-38).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,E,T", [(1, 128, 1, 1), (1, 2048, 64, 8), (3, 384, 5, 5), (13, 2048, 60, 4), (16, 1024, 128, 8),
                                     (127, 256, 64, 2), (129, 128, 8, 2), (300, 640, 17, 3), (5, 256, 1000, 32), (2, 128, 1024, 32),
                                     (65, 160 * 8, 250, 9), (512, 384, 130, 8), (40, 128, 1023, 4)])
def test_route(w, M, K, E, T, dtype):
    x, router, bias = make(M + K + E, M, K, E, dtype)
    check(w, x, router, T)
    check(w, x, router, T, score="sigmoid", bias=bias, scale=2.5)
    check(w, x, router, T, normalize=False, scale=0.5)


def test_ties_go_to_the_lowest_expert(w):
    x, router, _ = make(3, 9, 256, 40, "bf16")
    router[7] = router[30]
    router[11] = router[30]
    router[39] = router[0]
    check(w, x, router, 32)
    same = router[:1].expand(40, -1).contiguous()
    ids, weights = w.w4a16_route(x, same, 6)
    assert torch.equal(ids.long(), torch.arange(6, device=DEV).expand(9, 6))
    assert torch.equal(weights, torch.full_like(weights, float(torch.tensor(1 / 6, dtype=torch.float64))))


@pytest.mark.parametrize("M,E", [(3, 20), (130, 80)])
def test_products_beyond_fp32(w, M, E):
    """bf16 values whose products lie outside fp32's range, on either side."""
    x, router, _ = make(8, M, 256, E, "bf16")
    check(w, (x.float() * 1e25).bfloat16(), (router.float() * 1e25).bfloat16(), 4, normalize=False)
    ids, _ = w.w4a16_route((x.float() * 1e-30).bfloat16(), (router.float() * 1e-30).bfloat16(), 4)
    want, _ = su.route((x.float() * 1e-30).bfloat16().double(), (router.float() * 1e-30).bfloat16().double(), 4)
    assert torch.equal(ids.long(), want)


def test_rows_of_no_numbers_still_choose(w):
    x, router, _ = make(4, 4, 128, 12, "bf16")
    x[1] = float("nan")
    ids, weights = w.w4a16_route(x, router, 5)
    for m in range(4):
        row = ids[m].tolist()
        assert len(set(row)) == 5 and min(row) >= 0 and max(row) < 12
    want, ww = su.route(x[[0, 2, 3]].double(), router.double(), 5)
    assert torch.equal(ids[[0, 2, 3]].long(), want)


def test_more_rows_than_a_pass(w):
    x, router, _ = make(5, 16384 + 37, 128, 8, "fp16")
    check(w, x, router, 2)
