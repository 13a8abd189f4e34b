"""The router, the experts' layer and the draw of a token used together, and as programs use them:
captured and replayed, on other streams, by several threads, in one workspace."""

import threading

import pytest
import torch

import serve_util as su
import train_util as tu
from gpu_util import DEV

pytestmark = pytest.mark.gpu

K, F, V, E, T, G = 256, 128, 32768, 6, 2, 128


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


@pytest.fixture(scope="module")
def model(w):
    ex = su.Experts(w, 500, E, K, F, "bf16", G)
    head = tu.Weight(w, 600, K, V, "bf16", G)
    router, router64 = tu.normal(601, (E, K), "bf16", 0.1)
    return ex, head, router, router64


def norm(x):
    return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def step(w, model, ids, u, **how):
    """One decoding step: embedding, a layer of experts, the head, the draw."""
    ex, head, router, _ = model
    x = norm(w.w4a16_embedding(ids, head.packed, K, V, G))
    y, _, _ = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G, residual=x)
    logits = w.w4a16_gemm(norm(y), head.packed, V, G)
    return w.w4a16_sample(logits, u, **how) + (logits,)


@pytest.mark.parametrize("M", [1, 5, 40])
def test_decoding(w, model, M):
    """Every token of a short text is the one that its logits and number give in 64 bits, and the experts'
    layer within it what its definition gives."""
    ex, head, router, router64 = model
    gen = torch.Generator().manual_seed(M)
    ids = torch.randint(0, V, (M,), generator=gen, dtype=torch.int32).to(DEV)
    for how in (dict(temperature=0.8, top_k=20, top_p=0.9), dict(temperature=0.0), dict(top_p=0.95), dict(min_p=0.02)):
        x = norm(w.w4a16_embedding(ids, head.packed, K, V, G))
        y, chosen, weights = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G, residual=x)
        want, ww = su.route(x.double(), router64, T)
        assert torch.equal(chosen.long(), want)
        su.check_moe(y, su.moe(ex, x.double(), chosen, ww, "silu", x.double()), "bf16")
        u = torch.rand((M,), generator=gen).to(DEV)
        new, logprob, logits = step(w, model, ids, u, **how)
        want, lp = su.sample(logits, u, how.get("temperature", 1.0), how.get("top_k", 0), how.get("top_p", 1.0), how.get("min_p", 0.0))
        assert new.cpu().numpy().tolist() == want.tolist()
        ids = new


@pytest.mark.parametrize("M", [1, 16, 40])
def test_captured_and_replayed(w, model, M):
    gen = torch.Generator().manual_seed(7)
    ids = torch.randint(0, V, (M,), generator=gen, dtype=torch.int32).to(DEV)
    u = torch.rand((M,), generator=gen).to(DEV)
    how = dict(temperature=0.9, top_p=0.9)
    step(w, model, ids, u, **how)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(w, model, ids, u, **how)
    for seed in range(4):
        gen = torch.Generator().manual_seed(100 + seed)
        ids.copy_(torch.randint(0, V, (M,), generator=gen, dtype=torch.int32))
        u.copy_(torch.rand((M,), generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = step(w, model, ids, u, **how)           # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b)


def test_on_other_streams(w, model):
    gen = torch.Generator().manual_seed(3)
    runs = []
    for M in (1, 9, 33, 64):
        ids = torch.randint(0, V, (M,), generator=gen, dtype=torch.int32).to(DEV)
        runs.append((ids, torch.rand((M,), generator=gen).to(DEV)))
    want = [step(w, model, i, u, top_p=0.9) for i, u in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(3):
        got = []
        for s, (i, u) in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(step(w, model, i, u, top_p=0.9))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_host_threads_on_one_stream(w, model):
    gen = torch.Generator().manual_seed(4)
    runs = []
    for M in (1, 16, 40):
        ids = torch.randint(0, V, (M,), generator=gen, dtype=torch.int32).to(DEV)
        runs.append((ids, torch.rand((M,), generator=gen).to(DEV)))
    want = [step(w, model, i, u, top_k=30) for i, u in runs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        for _ in range(20):
            got = step(w, model, *runs[k], top_k=30)
            if not all(bool(torch.equal(a, b)) for a, b in zip(want[k], got)):
                wrong.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(runs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_one_workspace_for_all(w, model):
    """Calls of every entry point, in order, in one workspace whose contents are anything but its first 512
    bytes; these are zero again after each."""
    ex, head, router, _ = model
    shapes = [(M, E, T) for M in (1, 16, 40, 700)]
    need = max([w.w4a16_moe_layer_workspace_bytes(M, K, F, E, T, G) for M, _, _ in shapes]
               + [w.w4a16_sample_workspace_bytes(M, V) for M in (1, 64)] + [w.w4a16_workspace_bytes(40, K, V, G)])
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    ws[:512] = 0
    for M, _, _ in shapes + shapes[::-1]:
        x, _ = tu.normal(M, (M, K), "bf16")
        u = torch.rand((M,), device=DEV)
        want = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G)
        got = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert int(ws[:512].sum()) == 0
        logits = w.w4a16_gemm(x[:64].contiguous(), head.packed, V, G)
        u = u[:64].contiguous()
        want = w.w4a16_sample(logits, u, top_p=0.9)
        got = w.w4a16_sample(logits, u, top_p=0.9, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert int(ws[:512].sum()) == 0


def test_rows_behind_the_last_are_left(w, model):
    ex, head, router, _ = model
    for M in (1, 3, 16, 21):
        x, _ = tu.normal(M, (M, K), "bf16")
        y = torch.full((M + 8, K), 7.0, dtype=torch.bfloat16, device=DEV)
        ids = torch.full((M + 8, T), 77, dtype=torch.int32, device=DEV)
        weights = torch.full((M + 8, T), 7.0, device=DEV)
        w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G, y=y[:M], ids=ids[:M], weights=weights[:M])
        assert bool((y[M:] == 7).all()) and bool((ids[M:] == 77).all()) and bool((weights[M:] == 7).all())
        z = torch.randn((M, 30000), device=DEV)
        new, lp = torch.full((M + 8,), 77, dtype=torch.int32, device=DEV), torch.full((M + 8,), 7.0, device=DEV)
        w.w4a16_sample(z, torch.rand((M,), device=DEV), top_p=0.8, ids=new[:M], logprob=lp[:M])
        assert bool((new[M:] == 77).all()) and bool((lp[M:] == 7).all())


def test_a_row_of_no_numbers_stays_alone(w, model):
    """x of one row is infinite or no number: the other rows' results are what they are without it."""
    ex, _, router, _ = model
    for M in (4, 16, 24):
        x, _ = tu.normal(M, (M, K), "bf16")
        want, ids, _ = w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G)
        for bad in (float("inf"), float("nan")):
            x2 = x.clone()
            x2[2, 5] = bad
            y, ids2, _ = w.w4a16_moe_layer(x2, router, ex.gate_up, ex.down_packed, F, T, G)
            rest = [m for m in range(M) if m != 2]
            assert torch.equal(ids2[rest], ids[rest]) and torch.equal(y[rest], want[rest])
            assert not bool(torch.isfinite(y[2].float()).any())


def test_weights_of_no_number_stay_in_their_row(w, model):
    ex, _, _, _ = model
    for M in (3, 20):
        x, _ = tu.normal(M, (M, K), "bf16")
        ids = torch.tensor([[1, 4]] * M, dtype=torch.int32, device=DEV)
        weights = torch.full((M, 2), 0.5, device=DEV)
        want = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, F, G)
        weights[1, 0] = float("nan")
        y = w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, F, G)
        rest = [m for m in range(M) if m != 1]
        assert torch.equal(y[rest], want[rest]) and bool(torch.isnan(y[1].float()).all())


def test_a_vocabulary_past_32_bits_of_bytes(w):
    """Rows whose addresses pass 4 GiB."""
    V2, M = 40000, 6
    stride = 1 << 30                                  # elements: 2 GiB from row to row
    base = torch.empty((M - 1) * stride + V2, dtype=torch.bfloat16, device=DEV)
    z = base.as_strided((M, V2), (stride, 1))
    gen = torch.Generator().manual_seed(2)
    z.copy_((2 * torch.randn((M, V2), generator=gen)).to(torch.bfloat16))
    u = torch.rand((M,), generator=gen).to(DEV)
    for how in (dict(t=1.0), dict(k=9), dict(p=0.9)):
        ids, _ = w.w4a16_sample(z, u, temperature=how.get("t", 1.0), top_k=how.get("k", 0), top_p=how.get("p", 1.0))
        assert ids.tolist() == su.sample(z, u, **how)[0].tolist()


def test_no_rows(w, model):
    ex, _, router, _ = model
    x = torch.empty((0, K), dtype=torch.bfloat16, device=DEV)
    ids, weights = w.w4a16_route(x, router, T)
    assert ids.shape == (0, T) and weights.shape == (0, T)
    assert w.w4a16_moe(x, ids, weights, ex.gate_up, ex.down_packed, F, G).shape == (0, K)
    assert w.w4a16_moe_layer(x, router, ex.gate_up, ex.down_packed, F, T, G)[0].shape == (0, K)
    new, logprob = w.w4a16_sample(torch.empty((0, V), device=DEV), torch.empty((0,), device=DEV), top_p=0.9)
    assert new.shape == (0,) and logprob.shape == (0,)


def test_graphs_of_few_rows_side_by_side(w, model):
    """Two captured draws replayed on two streams at once, each with the workspace of its own graph."""
    z = torch.randn((2, 3, 40000), device=DEV)
    u = torch.rand((2, 3), device=DEV)
    want = [w.w4a16_sample(z[k], u[k], top_p=0.8) for k in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w.w4a16_sample(z[k], u[k], top_p=0.8))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k][0], want[k][0]) and torch.equal(outs[k][1], want[k][1])
