"""The draw of a token against its definition in 64 bits."""

import math

import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


def make(seed, M, V, dtype, spread=2.5, pad=0, banned=0.05):
    gen = torch.Generator().manual_seed(seed)
    z = spread * torch.randn((M, V + pad), generator=gen)
    likely = torch.randint(0, V, (M, 5), generator=gen)
    z.scatter_add_(1, likely, 8.0 * torch.rand((M, 5), generator=gen))
    z[torch.rand(z.shape, generator=gen) < banned] = -math.inf
    z[:, V // 2] = 0.0
    return z.to(su.dt(dtype)).to(DEV)[:, :V], torch.rand((M,), generator=gen).to(DEV)


def check(w, z, u, t=1.0, k=0, p=1.0, min_p=0.0):
    ids, logprob = w.w4a16_sample(z, u, temperature=t, top_k=k, top_p=p, min_p=min_p)
    want, lp = su.sample(z, u, t, k, p, min_p)
    assert np.array_equal(ids.cpu().numpy(), want), (ids.cpu().numpy(), want)
    got = logprob.double().cpu().numpy()
    fine = np.isfinite(lp)
    assert np.array_equal(fine, np.isfinite(got))
    # one rounding to fp32 (half a step: 2^-24); sums of up to 2^18 terms in fp64 below 1e-10
    assert (np.abs(got[fine] - lp[fine]) <= 2.0 ** -24 * np.abs(lp[fine]) * 1.001 + 1e-10).all()


SETTINGS = [dict(), dict(t=0.0), dict(t=0.7, k=1), dict(k=20), dict(k=1000), dict(p=0.9), dict(t=1.7, p=0.99), dict(p=1e-6), dict(min_p=0.05),
            dict(t=0.6, k=50, p=0.8), dict(k=50, p=0.95, min_p=0.1), dict(p=0.7, min_p=0.01), dict(k=10 ** 6, p=2.0, min_p=-1.0),
            dict(p=0.0), dict(min_p=1.0), dict(min_p=7.0), dict(t=50.0, p=0.5)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (2, 7), (5, 64), (4, 257), (3, 1000), (2, 8191), (2, 8193), (3, 32003), (2, 131072)])
def test_sample(w, M, V, dtype):
    z, u = make(M + V, M, V, dtype)
    for s in SETTINGS:
        check(w, z, u, **s)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", [(64, 24600), (65, 24600), (3, 49155), (130, 9001)])
def test_few_rows_and_many(w, M, V, dtype):
    """Rows that take several workgroups each, and rows that take one."""
    z, u = make(M, M, V, dtype, spread=1.0)
    for s in SETTINGS:
        check(w, z, u, **s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad", [1, 5, 8])
def test_rows_with_a_stride(w, pad, dtype):
    z, u = make(pad, 6, 1003, dtype, pad=pad)
    assert z.stride(0) == 1003 + pad
    for s in SETTINGS[:10]:
        check(w, z, u, **s)
    check(w, z[:, 3:], u, k=7, p=0.9)            # rows that begin inside 16 bytes


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_settings_of_each_row(w, dtype):
    M = 40
    z, u = make(77, M, 5003, dtype)
    gen = torch.Generator().manual_seed(1)
    t = torch.rand((M,), generator=gen) * 1.5
    t[::7] = 0.0
    k = torch.randint(-3, 60, (M,), generator=gen, dtype=torch.int32)
    p = torch.rand((M,), generator=gen) * 1.3
    m = torch.rand((M,), generator=gen) * 0.2 - 0.05
    check(w, z, u, t.to(DEV), k.to(DEV), p.to(DEV), m.to(DEV))
    check(w, z, u, 0.8, k.to(DEV), 0.9, m.to(DEV))
    check(w, z, u, t.to(DEV), 30, p.to(DEV), 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_at_every_threshold(w, dtype):
    """Few distinct values: thresholds fall among equals, the lowest indices stay."""
    gen = torch.Generator().manual_seed(5)
    for V in (96, 9001, 20000):
        z = torch.randint(0, 3, (8, V), generator=gen).float().to(su.dt(dtype)).to(DEV)
        u = torch.rand((8,), generator=gen).to(DEV)
        for k in (1, 5, V // 3, V - 1):
            check(w, z, u, k=k)
            check(w, z, u, k=k, p=0.37)
        for p in (0.01, 0.31, 0.62, 0.999):
            check(w, z, u, p=p)
        same = torch.zeros((2, V), device=DEV).to(su.dt(dtype))
        check(w, same, torch.tensor([0.0, 0.9999999], device=DEV), k=V // 2, p=0.31)
        check(w, same, torch.tensor([0.5, 0.25], device=DEV))


def test_zeros_of_either_sign_tie(w):
    z = torch.full((1, 64), -5.0, device=DEV)
    z[0, 10], z[0, 20] = -0.0, 0.0
    for k in (1, 2):
        check(w, z, torch.tensor([0.6], device=DEV), k=k)
    ids, _ = w.w4a16_sample(z, torch.tensor([0.6], device=DEV), temperature=0.0)
    assert int(ids) == 10


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_infinities_and_no_numbers(w, dtype):
    z, u = make(9, 7, 3001, dtype)
    z = z.clone()
    z[0, :] = -math.inf                          # nothing
    z[1, :] = math.nan                           # nothing
    z[2, ::2] = math.nan
    z[3, [5, 900, 2000]] = math.inf              # these alone
    z[4, :] = -math.inf
    z[4, 2999] = -3.0                            # one
    z[5, 0] = math.nan
    for s in SETTINGS:
        check(w, z, u, **s)
    ids, logprob = w.w4a16_sample(z, u)
    assert ids[:2].tolist() == [-1, -1] and logprob[:2].tolist() == [-math.inf] * 2 and int(ids[4]) == 2999
    assert float(logprob[4]) == 0.0 and int(ids[3]) in (5, 900, 2000)


@pytest.mark.parametrize("V", [50, 4099, 40000])
def test_numbers_at_the_ends(w, V):
    z, _ = make(V, 6, V, "fp32")
    z = z.clone()
    z[:, 0], z[:, -1] = -math.inf, -math.inf
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 2.0 ** -24, 1.0, -1.0, math.nan], device=DEV)
    for s in (dict(), dict(k=9), dict(p=0.8), dict(t=0.05)):
        check(w, z, u, **s)


@pytest.mark.parametrize("M,V", [(4, 3001), (3, 40000), (70, 26000)])
def test_extreme_temperatures_and_logits(w, M, V):
    z, u = make(V, M, V, "fp32")
    for t in (1e-42, 1e-20, 1e-3, 1e4, 1e30, math.inf, math.nan, -1.0):
        for how in (dict(), dict(p=0.6), dict(k=30, p=0.6)):
            check(w, z, u, t=t, **how)
    for lift in (1e4, -3e38):
        far = (z + lift).clamp(min=-3.4e38)
        for how in (dict(), dict(p=0.9), dict(k=30), dict(min_p=0.1)):
            check(w, far, u, **how)


@pytest.mark.parametrize("p", [0.5, 0.999, 1.0 - 2.0 ** -24, 2.0 ** -149])
@pytest.mark.parametrize("M,V", [(2, 40000), (2, 9000), (90, 24580)])
def test_top_p_at_its_ends(w, M, V, p):
    """Weights that all lie far below the largest count in the sum that p is reached in."""
    z = torch.full((M, V), -26.0, device=DEV)
    z[:, V // 3] = 0.0
    z[:, V // 2:V // 2 + 7] = -1.0
    check(w, z, torch.rand((M,), generator=torch.Generator().manual_seed(1)).to(DEV), p=p)
    z, u = make(V, M, V, "fp32", spread=6.0)
    check(w, z, u, p=p)


def test_every_token_by_its_share(w):
    """u on a grid: each token as often as its weight says."""
    z = torch.tensor([[0.0, math.log(3.0), -math.inf, math.log(4.0)]], device=DEV).expand(800, 4)
    u = ((torch.arange(800, device=DEV) + 0.5) / 800).float()
    ids, _ = w.w4a16_sample(z.contiguous(), u)
    assert torch.bincount(ids, minlength=4).tolist() == [100, 300, 0, 400]


def test_one_row_for_many_draws(w):
    """Rows may be the same memory: a stride of 0 is refused, a copy is not."""
    z, u = make(3, 1, 500, "bf16")
    with pytest.raises(ValueError):
        w.w4a16_sample(z.expand(4, 500), u.expand(4).contiguous())


@pytest.mark.parametrize("spread", [0.001, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_flat_and_steep_rows(w, spread, dtype):
    z, u = make(21, 3, 70001, dtype, spread=spread, banned=0.0)
    for s in SETTINGS:
        check(w, z, u, **s)
