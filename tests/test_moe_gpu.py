"""The experts' layer against its definition in 64 bits."""

import pytest
import torch

import serve_util as su
import train_util as tu
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


_experts = {}


def experts(w, *key):
    if key not in _experts:
        _experts.clear()               # one at a time
        _experts[key] = su.Experts(w, 100, *key)
    return _experts[key]


def entries(seed, M, E, T, drop=0.0):
    gen = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(max(E, T), generator=gen)[:T] % E for _ in range(M)]).to(torch.int32)
    ids[torch.rand((M, T), generator=gen) < drop] = -1
    weights = torch.softmax(torch.randn((M, T), generator=gen), 1)
    return ids.to(DEV), weights.to(DEV)


def run(w, ex, M, T, act="silu", drop=0.0, residual=True, seed=0, ids=None, weights=None):
    x, x64 = tu.normal(seed + M, (M, ex.K), ex.dtype)
    if ids is None:
        ids, weights = entries(seed + M, M, ex.E, T, drop)
    r, r64 = tu.normal(seed + M + 1, (M, ex.K), ex.dtype) if residual else (None, None)
    y = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G, act=act, residual=r)
    su.check_moe(y, su.moe(ex, x64, ids, weights.double(), act, r64), ex.dtype)
    return y


ROWS = [1, 2, 13, 16, 17, 40, 77, 200]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype,K,F,G", [("bf16", 512, 256, 128), ("fp16", 512, 256, 128), ("bf16", 256, 384, 64), ("fp16", 384, 128, 32),
                                         ("bf16", 256, 256, -1), ("fp16", 1024, 640, 64), ("bf16", 256, 128, 32)])
def test_moe(w, M, dtype, K, F, G):
    ex = experts(w, 6, K, F, dtype, G)
    run(w, ex, M, 2, seed=K)
    run(w, ex, M, 3, act="gelu", drop=0.3, residual=False, seed=K)
    run(w, ex, M, 1, act="gelu_tanh", seed=F)


@pytest.mark.parametrize("M", [1, 5, 16, 17, 96])
def test_many_experts(w, M):
    ex = experts(w, 70, 128, 128, "bf16", 128)
    run(w, ex, M, 8)
    run(w, ex, M, 32, drop=0.5)


@pytest.mark.parametrize("K,F,G,dtype", [(4096, 128, 32, "bf16"), (4096, 256, 64, "fp16"), (4224, 128, 128, "bf16"), (2176, 384, 128, "fp16")])
def test_long_rows(w, K, F, G, dtype):
    ex = experts(w, 3, K, F, dtype, G)
    for M in (1, 9, 16, 18):
        run(w, ex, M, 2, seed=K)


@pytest.mark.parametrize("M", [1, 16, 33, 150])
def test_one_expert_and_one_entry(w, M):
    ex = experts(w, 1, 256, 128, "fp16", 128)
    run(w, ex, M, 1)
    run(w, ex, M, 4)                   # the same expert four times: all weights count


@pytest.mark.parametrize("M", [1, 7, 16, 20, 70])
def test_entries_that_name_no_expert(w, M):
    ex = experts(w, 6, 512, 256, "bf16", 128)
    weights = torch.rand((M, 3), device=DEV)
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((M, 3), bad, dtype=torch.int32, device=DEV)
        x, _ = tu.normal(1, (M, 512), "bf16")
        y = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G)
        assert torch.equal(y, torch.zeros_like(y))
        r, _ = tu.normal(2, (M, 512), "bf16")
        y = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G, residual=r)
        assert torch.equal(y, r)
        ids[M // 2, 1] = 4             # a lone entry
        run(w, ex, M, 3, ids=ids, weights=weights)


@pytest.mark.parametrize("M", [3, 16, 50])
def test_one_expert_takes_all(w, M):
    ex = experts(w, 6, 512, 256, "bf16", 128)
    ids = torch.full((M, 2), 5, dtype=torch.int32, device=DEV)
    ids[:, 1] = 0
    run(w, ex, M, 2, ids=ids, weights=torch.rand((M, 2), device=DEV))


@pytest.mark.parametrize("M", [4, 40])
def test_strided_experts_and_residual_in_place(w, M):
    ex = su.Experts(w, 300, 3, 256, 128, "bf16", 128, 48)
    assert ex.gate_up.stride(0) % 16 == 0
    ids, weights = entries(8, M, 3, 2)
    x, x64 = tu.normal(9, (M, 256), "bf16")
    y, r64 = tu.normal(10, (M, 256), "bf16")
    out = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G, residual=y, y=y)
    assert out.data_ptr() == y.data_ptr()
    su.check_moe(y, su.moe(ex, x64, ids, weights.double(), "silu", r64), "bf16")
    # every other expert of a larger stack
    alone = w.w4a16_moe(x, ids % 2, weights, ex.gate_up[::2], ex.down_packed[::2], ex.F, ex.G)
    pick = torch.tensor([0, 2], device=DEV)[(ids % 2).long()].to(torch.int32)
    su.check_moe(alone, su.moe(ex, x64, pick, weights.double()), "bf16")


@pytest.mark.parametrize("M", [1, 12, 60])
def test_same_bits_every_time(w, M):
    ex = experts(w, 6, 512, 256, "bf16", 128)
    x, _ = tu.normal(11, (M, 512), "bf16")
    ids, weights = entries(12, M, 6, 4)
    first = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G)
    for _ in range(5):
        assert torch.equal(first, w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G))


@pytest.mark.parametrize("M", [1, 16, 80])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_layer(w, M, score):
    ex = experts(w, 6, 512, 256, "bf16", 128)
    x, x64 = tu.normal(13, (M, 512), "bf16")
    router, router64 = tu.normal(14, (6, 512), "bf16", 0.05)
    r, r64 = tu.normal(15, (M, 512), "bf16")
    y, ids, weights = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, ex.F, 2, ex.G, score=score, scale=1.5, residual=r)
    want, ww = su.route(x64, router64, 2, score=score, scale=1.5)
    assert torch.equal(ids.long(), want)
    su.check_moe(y, su.moe(ex, x64, ids, ww, "silu", r64), "bf16")
    ids2, weights2 = w.w4a16_route(x, router, 2, score=score, scale=1.5)
    assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
    assert torch.equal(y, w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G, residual=r))


def test_large_values_keep_their_range(w):
    """h beyond fp16's range, as bf16 models have it."""
    ex = experts(w, 6, 512, 256, "bf16", 128)
    for M in (2, 30):
        x, x64 = tu.normal(16, (M, 512), "bf16", 300.0)
        ids, weights = entries(17, M, 6, 2)
        ref = su.moe(ex, x64, ids, weights.double())
        assert float(tu.gated(ex.up[0], ex.F, x64, "silu").abs().max()) > 65504
        su.check_moe(w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, ex.F, ex.G), ref, "bf16")


def test_more_rows_than_a_pass(w):
    ex = experts(w, 3, 128, 128, "bf16", 128)
    run(w, ex, 2 * 512 + 5, 32)        # 16384 / 32 rows a pass


@pytest.mark.parametrize("M", [2, 16, 40])
def test_experts_past_32_bits_of_bytes(w, M):
    """Experts whose offsets pass 4 GiB."""
    ex = su.Experts(w, 700, 3, 256, 128, "bf16", 128)
    stride = 3 << 30

    def spread(packed):
        n = packed.shape[1]
        far = torch.empty(2 * stride + n, dtype=torch.uint8, device=DEV).as_strided((3, n), (stride, 1))
        far.copy_(packed)
        return far
    ids, weights = entries(3, M, 3, 2)
    x, x64 = tu.normal(4, (M, 256), "bf16")
    y = w.w4a16_moe(x, ids, weights, spread(ex.gate_up), spread(ex.down_packed), ex.F, ex.G)
    su.check_moe(y, su.moe(ex, x64, ids, weights.double()), "bf16")
