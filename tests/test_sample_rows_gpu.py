"""The draw of more rows than a launch's 2^32 threads hold as workgroups."""

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


@pytest.mark.parametrize("M", [(1 << 20) + 5, (1 << 22) + 3])
def test_more_rows_than_a_launch(w, M):
    gen = torch.Generator(device=DEV).manual_seed(6)
    z = torch.randint(-3, 4, (M, 2), generator=gen, device=DEV).float()
    u = torch.rand((M,), generator=gen, device=DEV)
    t = torch.rand((M,), generator=gen, device=DEV) + 0.5
    t[torch.rand((M,), generator=gen, device=DEV) < 0.25] = 0.0
    k = torch.randint(0, 3, (M,), generator=gen, device=DEV, dtype=torch.int32)
    ids, logprob = w.w4a16_sample(z, u, temperature=t, top_k=k, top_p=torch.ones_like(t), min_p=torch.zeros_like(t))
    z64, t64 = z.double(), t.double()
    weight = torch.exp((z64 - z64.max(1, keepdim=True).values) / torch.where(t64 > 0, t64, torch.ones_like(t64))[:, None])
    first = (z[:, 0] >= z[:, 1]).long()                    # 1: the largest is entry 0, also of two equal ones
    one = (t <= 0) | (k == 1)
    alone = torch.stack([first, 1 - first], 1).double()
    weight = torch.where(one[:, None], alone, weight)
    total = weight.sum(1)
    want = torch.where(weight[:, 0] > u.double() * total, 0, 1)
    assert torch.equal(ids.long(), want)
    lp = torch.log(weight.gather(1, want[:, None])[:, 0] / total)
    # one rounding to fp32 (half a step: 2^-24), the rest in fp64
    assert ((logprob.double() - lp).abs() <= 2.0 ** -24 * lp.abs() * 1.001 + 1e-10).all()


def test_long_rows_in_the_last_launch(w):
    """The rows left for the last launch are few and of a length that a call of so few takes several launches for."""
    M, V = (1 << 20) + 3, 24577
    assert w.w4a16_sample_workspace_bytes(M, V) == 0 < w.w4a16_sample_workspace_bytes(3, V)
    z = torch.zeros((M, V), dtype=torch.float16, device=DEV)
    at = (torch.arange(M, device=DEV) * 977) % V
    z.scatter_(1, at[:, None], 40.0)
    u = torch.full((M,), 0.5, device=DEV)
    ids, _ = w.w4a16_sample(z, u, top_p=0.9, workspace=torch.zeros(512, dtype=torch.uint8, device=DEV))
    assert torch.equal(ids.long(), at)
