"""The draw of few long rows, which takes several launches and a workspace: rows of every kind side by side, in a
workspace that holds no numbers, so that a field which no launch has written shows."""

import math

import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import DEV

pytestmark = pytest.mark.gpu

SIZES = [(40, 40000), (100, 65600), (3, 131072)]


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


def make(seed, M, V, dtype, spread=2.5):
    gen = torch.Generator().manual_seed(seed)
    z = spread * torch.randn((M, V), generator=gen)
    likely = torch.randint(0, V, (M, 5), generator=gen)
    z.scatter_add_(1, likely, 8.0 * torch.rand((M, 5), generator=gen))
    z[torch.rand(z.shape, generator=gen) < 0.05] = -math.inf
    return z.to(su.dt(dtype)).to(DEV), torch.rand((M,), generator=gen).to(DEV)


def check(w, z, u, t=1.0, k=0, p=1.0, min_p=0.0):
    need = w.w4a16_sample_workspace_bytes(*z.shape)
    assert need > 512
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    ws[:512] = 0
    ids, logprob = w.w4a16_sample(z, u, temperature=t, top_k=k, top_p=p, min_p=min_p, workspace=ws)
    if isinstance(t, torch.Tensor):
        # +infinity excludes all others at any temperature; in the definition -infinity over an infinite one is no number
        t = torch.where((z == math.inf).any(dim=1) & (t == math.inf), torch.ones_like(t), t)
    want, lp = su.sample(z, u, t, k, p, min_p)
    assert np.array_equal(ids.cpu().numpy(), want), (ids.cpu().numpy(), want)
    got = logprob.double().cpu().numpy()
    fine = np.isfinite(lp)
    assert np.array_equal(fine, np.isfinite(got))
    # one rounding to fp32 (half a step: 2^-24); sums of up to 2^18 terms in fp64 below 1e-10
    assert (np.abs(got[fine] - lp[fine]) <= 2.0 ** -24 * np.abs(lp[fine]) * 1.001 + 1e-10).all()
    assert int(ws[:512].sum()) == 0


def each_row(values, M, dtype):
    return torch.tensor([values[m % len(values)] for m in range(M)], dtype=dtype, device=DEV)


def settings(M, V):
    """Lists of lengths without a common divisor: the kinds of rows meet in every order."""
    return dict(t=each_row([1.0, 0.0, 0.7, 1.6, math.inf, 0.9, -1.0], M, torch.float32),
                k=each_row([0, 1, 50, 192, 193, 1000, 1024, 1025, 2000, V, -5], M, torch.int32),
                p=each_row([1.0, 0.9, 0.5, 1e-6, 2.0], M, torch.float32),
                min_p=each_row([0.0, 0.02, -1.0, 0.3], M, torch.float32))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", SIZES)
def test_rows_of_every_kind(w, M, V, dtype):
    z, u = make(M + V, M, V, dtype)
    s = settings(M, V)
    check(w, z, u, **s)
    for name, one in (("t", 0.8), ("k", 0), ("k", 300), ("p", 0.9), ("p", 1.0), ("min_p", 0.0)):
        check(w, z, u, **{**s, name: one})
    for k in (192, 193, 1000, 1024, 1025, 5000, V - 1):
        check(w, z[:4], u[:4], t=0.9, k=k)
        check(w, z[:4], u[:4], k=k, p=0.8, min_p=0.001)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", SIZES)
def test_infinities_and_no_numbers(w, M, V, dtype):
    z, u = make(M, M, V, dtype)
    s = settings(M, V)
    for kind in range(6):
        bad = z.clone()
        for m in range(kind % 2, M, 2):
            if kind // 2 == 0:
                bad[m] = -math.inf if m % 4 < 2 else math.nan                # nothing to draw
            elif kind // 2 == 1:
                bad[m, [5, V // 2, V - 2]] = math.inf                        # these alone
            else:
                bad[m, ::2] = math.nan
                bad[m, 1] = -math.inf
        check(w, bad, u, **s)
        for one in (dict(), dict(t=0.0), dict(k=3), dict(k=50, p=0.9), dict(k=500), dict(k=2000, p=0.9), dict(p=0.9), dict(p=0.7, min_p=0.01)):
            check(w, bad[:5], u[:5], **one)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", SIZES)
def test_ties_at_every_threshold(w, M, V, dtype):
    """Few distinct values: thresholds fall among equals, the lowest indices stay; lists run over."""
    gen = torch.Generator().manual_seed(V)
    z = torch.randint(0, 3, (M, V), generator=gen).float().to(su.dt(dtype)).to(DEV)
    u = torch.rand((M,), generator=gen).to(DEV)
    check(w, z, u, **settings(M, V))
    for k in (1, 5, 192, 193, 1000, V // 3, V - 1):
        check(w, z[:4], u[:4], k=k)
        check(w, z[:4], u[:4], k=k, p=0.37)
    for p in (0.01, 0.31, 0.62, 0.999):
        check(w, z[:4], u[:4], p=p)
    same = torch.zeros((4, V), device=DEV).to(su.dt(dtype))
    check(w, same, u[:4] if M >= 4 else torch.rand((4,), generator=gen).to(DEV), k=V // 2, p=0.31)


@pytest.mark.parametrize("k", [0, 192, 193, 1000, 5000])
def test_few_tokens_that_can_be_drawn(w, k):
    """Fewer finite logits than k; all of them at one end of the row."""
    M, V = 6, 40000
    z = torch.full((M, V), -math.inf, device=DEV)
    for m, n in enumerate((1, 2, 100, 191, 600, 3000)):
        at = slice(0, n) if m % 2 else slice(V - n, V)
        z[m, at] = torch.randn((n,), generator=torch.Generator().manual_seed(n)).to(DEV)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.3, 0.6, 0.9, 0.1], device=DEV)
    check(w, z, u, k=k)
    check(w, z, u, k=k, p=0.8)


@pytest.mark.parametrize("M,V", [(6, 40000), (6, 5000)])
def test_settings_of_no_number(w, M, V):
    """A temperature that is no number draws the largest; a top_p or min_p that is none limits nothing."""
    z, u = make(V, M, V, "bf16")
    none = math.nan
    for s in (dict(t=none), dict(p=none), dict(min_p=none), dict(k=40, p=none), dict(p=0.8, min_p=none),
              dict(t=each_row([none, 0.7], M, torch.float32), p=each_row([0.9, none, 1.0], M, torch.float32), min_p=each_row([none, 0.1], M, torch.float32))):
        ids, _ = w.w4a16_sample(z, u, temperature=s.get("t", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0), min_p=s.get("min_p", 0.0))
        assert np.array_equal(ids.cpu().numpy(), su.sample(z, u, **s)[0])
