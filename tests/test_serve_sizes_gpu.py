"""The router, the experts' layer and the draw of a token at the ends of their ranges of sizes."""

import numpy as np
import pytest
import torch

import serve_util as su
import train_util as tu
from gpu_util import DEV, TORCH_DTYPE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,E,T", [(3, 2176, 5, 2), (1, 8320, 64, 8), (2, 131072, 17, 3), (2, 1 << 20, 3, 2), (130, 6272, 80, 4), (600, 4096, 20, 3),
                                     (33, 2176, 1024, 32)])
def test_route_of_long_rows(w, M, K, E, T, dtype):
    """K beyond what a lane holds of an expert's weights, and beyond one batch of loads of a tile's waves."""
    gen = torch.Generator().manual_seed(M + K)
    x = torch.randn((M, K), generator=gen).to(TORCH_DTYPE[dtype]).to(DEV)
    router = (torch.randn((E, K), generator=gen) * 1.5 / K ** 0.5).to(TORCH_DTYPE[dtype]).to(DEV)
    bias = (torch.randn((E,), generator=gen) * 0.1).to(DEV)
    for how in (dict(), dict(score="sigmoid", bias=bias, scale=2.5), dict(normalize=False)):
        ids, weights = w.w4a16_route(x, router, T, **how)
        want, ww = [], []
        for m0 in range(0, M, 100):
            a, b = su.route(x[m0:m0 + 100].double(), router.double(), T, **how)
            want.append(a)
            ww.append(b)
        want, ww = torch.cat(want), torch.cat(ww)
        assert torch.equal(ids.long(), want)
        # one rounding to fp32 (half a step: 2^-24), the rest in fp64
        assert ((weights.double() - ww).abs() <= 2.0 ** -24 * ww.abs() * 1.001 + 1e-38).all()


@pytest.mark.parametrize("M,T", [(1, 16), (16, 16), (1, 32), (17, 16), (300, 16)])
def test_as_many_experts_as_there_may_be(w, M, T):
    """1024 experts, eight different ones: expert e has the weights of e % 8."""
    ex = su.Experts(w, 40, 8, 256, 128, "bf16", 128)
    up, down = ex.gate_up.repeat(128, 1), ex.down_packed.repeat(128, 1)
    gen = torch.Generator().manual_seed(M)
    ids = torch.stack([torch.randperm(1024, generator=gen)[:T] for _ in range(M)]).to(torch.int32)
    ids[0, 0], ids[M - 1, T - 1] = 1023, 1024
    ids, weights = ids.to(DEV), torch.rand((M, T), generator=gen).to(DEV)
    x, x64 = tu.normal(M, (M, 256), "bf16")
    y = w.w4a16_moe(x, ids, weights, up, down, 128, 128)
    su.check_moe(y, su.moe(ex, x64, torch.where(ids < 1024, ids % 8, ids), weights.double()), "bf16")


@pytest.mark.parametrize("K,F", [(128, 1 << 15), (1 << 15, 128)])
def test_the_widest_layers(w, K, F):
    """h's rows, or those of x, up to the end of the 32 bits that address a pass of 16384 entries."""
    ex = su.Experts(w, 60, 2, K, F, "bf16", 128)
    for M, T in ((1, 2), (16, 2), (515, 32)):
        gen = torch.Generator().manual_seed(M)
        ids = torch.randint(-1, 2, (M, T), generator=gen, dtype=torch.int32).to(DEV)
        ids[M - 1] = 1
        weights = torch.softmax(torch.randn((M, T), generator=gen), 1).to(DEV)
        x, x64 = tu.normal(M, (M, K), "bf16")
        y = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, F, 128)
        su.check_moe(y, su.moe(ex, x64, ids, weights.double()), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_draw_from_millions(w, dtype):
    V = 3000017
    gen = torch.Generator().manual_seed(1)
    z = (2.5 * torch.randn((1, V), generator=gen)).to(su.dt(dtype)).to(DEV)
    u = torch.rand((1,), generator=gen).to(DEV)
    for how in (dict(), dict(t=0.0), dict(k=50, p=0.9), dict(p=0.95), dict(k=1000), dict(k=5000, p=0.5), dict(min_p=0.01)):
        ids, logprob = w.w4a16_sample(z, u, temperature=how.get("t", 1.0), top_k=how.get("k", 0), top_p=how.get("p", 1.0),
                                      min_p=how.get("min_p", 0.0))
        want, lp = su.sample(z, u, **how)
        assert np.array_equal(ids.cpu().numpy(), want)
        # one rounding to fp32 (half a step: 2^-24); sums of up to 2^22 terms in fp64 below 2e-9
        assert np.abs(logprob.double().cpu().numpy() - lp) <= 2.0 ** -24 * np.abs(lp) * 1.001 + 2e-9


def test_draw_from_the_longest_row(w):
    """2^28 logits: one that holds nearly all the weight, first, inside or last."""
    V = 1 << 28
    z = torch.zeros((1, V), dtype=torch.float16, device=DEV)
    u = torch.tensor([0.5], device=DEV)
    for at in (0, 123456789, V - 1):
        z[0, at] = 40.0
        for how in (dict(), dict(temperature=0.0), dict(top_k=5), dict(top_k=1), dict(top_p=0.9), dict(min_p=0.5)):
            ids, logprob = w.w4a16_sample(z, u, **how)
            assert int(ids) == at and float(logprob) > -1e-3
        z[0, at] = 0.0


@pytest.mark.parametrize("V", [1 << 20, (1 << 22) + 5])
def test_draw_from_a_long_flat_row(w, V):
    """All logits the same: the token is at u of what the thresholds leave, which are the first."""
    z = torch.zeros((1, V), dtype=torch.bfloat16, device=DEV)
    for share in (0.25, 0.5):
        u = torch.tensor([share], device=DEV)
        for how, kept in ((dict(), V), (dict(top_k=V // 2), V // 2), (dict(top_k=999), 999), (dict(top_p=0.5), (V + 1) // 2)):
            ids, logprob = w.w4a16_sample(z, u, **how)
            assert int(ids) == int(share * kept)               # the first v with v + 1 > share kept
            assert abs(float(logprob) + np.log(kept)) <= 2.0 ** -24 * np.log(kept) * 1.001 + 1e-10
