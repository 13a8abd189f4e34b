"""The training and scoring operators against their definitions in 64 bits.

Tolerances count roundings, each at most half a step relative to its value (ULP below):
an output is rounded once; a gradient's product also takes W rounded to the operand type
and, where the operator forms it, the inner gradient rounded to bf16. Roundings of
independent terms add up in the norm to less than their sum, so a gradient row is held to
(number of roundings) x ULP in the norm. Losses are fp32: a logit's error is taken as
2^-24 sqrt(128 + K/128) 143 s_max |x|_2, the random-sign growth of the rounding of a sum
of 128-term blocks whose terms are at most (128 + 15) s_max |x_k|, and the loss's as
twice that plus 2^-20 of itself (exp, log, sums of V terms)."""

import numpy as np
import pytest
import torch

import synth
import train_util as tu
from gpu_util import DEV
from train_util import ULP, norm_err, normal

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


@pytest.fixture(scope="module")
def w():
    import w4a16_int4_weight_amd as mod
    return mod


_weights = {}


def weight(w, K, N, dtype, G, seed=7000):
    key = (K, N, dtype, G, seed)
    if key not in _weights:
        if len(_weights) > 6:
            _weights.clear()
        _weights[key] = tu.Weight(w, seed, K, N, dtype, G)
    return _weights[key]


def logit_eps(x64, K):
    return 2.0 ** -24 * np.sqrt(128 + K / 128) * 143 * 0.02 * x64.norm(dim=1)


def rows_within(got, ref, tol, what):
    assert torch.isfinite(got.float()).all(), what
    err = (got.double() - ref).norm(dim=1)
    lim = tol * ref.norm(dim=1) + 1e-30
    bad = (err > lim).nonzero().flatten()
    assert bad.numel() == 0, f"{what}: rows {bad[:8].tolist()}, worst {float((err / lim).max()):.2f} of the tolerance"


# ------------------------------------------------------------------ dx = dy W^T

@pytest.mark.parametrize("M,K,N,dtype,G", [
    (1, 128, 8, "bf16", 128), (1, 256, 24, "fp16", 128), (3, 384, 72, "bf16", -1), (16, 512, 520, "fp16", 64),
    (17, 256, 1000, "bf16", 32), (33, 640, 136, "bf16", 128), (64, 1024, 2048, "fp16", 256), (65, 384, 264, "bf16", 128),
    (128, 2048, 512, "bf16", 128), (129, 256, 4104, "fp16", 128), (257, 896, 1096, "bf16", 64), (300, 2048, 2056, "bf16", 128),
    (1030, 512, 640, "fp16", 32),
])
def test_gemm_grad(w, M, K, N, dtype, G):
    print(f"gemm_grad M={M} K={K} N={N} {dtype} G={G}", flush=True)
    wt = weight(w, K, N, dtype, G)
    dy, dy64 = normal(M * 31 + N, (M, N), dtype)
    dx = w.w4a16_gemm_grad(dy, wt.packed, K, G)
    torch.cuda.synchronize()
    rows_within(dx, dy64 @ wt.dev64.t(), 2 * ULP[dtype], "dx")
    again = w.w4a16_gemm_grad(dy, wt.packed, K, G)
    assert torch.equal(dx.view(torch.int16), again.view(torch.int16))


def test_gemm_grad_one_hot_is_the_gather(w):
    # dy a row of the identity: dx is column n of W rounded once, what the gather returns
    K, N, G = 512, 136, 64
    wt = weight(w, K, N, "fp16", G)
    dy = torch.eye(N, dtype=torch.float16, device=DEV)
    dx = w.w4a16_gemm_grad(dy, wt.packed, K, G)
    e = w.w4a16_embedding(torch.arange(N, dtype=torch.int32, device=DEV), wt.packed, K, N, G, torch.float16)
    assert torch.equal(dx, e)


def test_gemm_grad_rows_do_not_mix(w):
    # a row of NaN, rows of infinities: only their own outputs; a tail stage past N reads
    # nothing of the next row
    K, N = 256, 88
    wt = weight(w, K, N, "bf16", 128)
    dy, dy64 = normal(5, (40, N), "bf16")
    clean = w.w4a16_gemm_grad(dy, wt.packed, K, 128)
    dirty = dy.clone()
    dirty[7] = float("nan")
    dirty[21] = float("inf")
    out = w.w4a16_gemm_grad(dirty, wt.packed, K, 128)
    keep = [m for m in range(40) if m not in (7, 21)]
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert torch.isnan(out[7]).all()


# ------------------------------------------------------------------ gated block

GATED = [
    (1, 128, 8, "bf16", 128, "silu"), (1, 2048, 6656, "bf16", 128, "silu"), (2, 256, 24, "fp16", 64, "gelu"),
    (5, 384, 136, "bf16", 32, "gelu_tanh"), (13, 2048, 1032, "fp16", 128, "gelu_tanh"), (16, 1024, 520, "bf16", -1, "silu"),
    (17, 512, 264, "bf16", 128, "gelu"), (33, 256, 1000, "fp16", 128, "silu"), (64, 1024, 512, "bf16", 64, "silu"),
    (65, 640, 328, "fp16", 32, "gelu"), (100, 2048, 2728, "bf16", 128, "silu"), (513, 512, 1096, "bf16", 128, "gelu_tanh"),
]


@pytest.mark.parametrize("M,K,F,dtype,G,act", GATED)
def test_gated(w, M, K, F, dtype, G, act):
    print(f"gated M={M} K={K} F={F} {dtype} G={G} {act}", flush=True)
    wt = weight(w, K, 2 * F, dtype, G)
    x, x64 = normal(M * 7 + F, (M, K), dtype)
    h = w.w4a16_gated(x, wt.packed, F, G, act=act)
    torch.cuda.synchronize()
    g, u = x64 @ wt.dev64[:, :F], x64 @ wt.dev64[:, F:]
    a = tu.act(act, g)
    ref = a * u
    # one rounding of h, and the fp32 errors of g, u (|a'| <= 1.13) and of exp
    slack = logit_eps(x64, K)[:, None] * (1.13 * u.abs() + a.abs()) + 2.0 ** -20 * (g * u).abs()
    worst = ((h.double() - ref).abs() / (ULP[dtype] * ref.abs() + slack + 2.0 ** -25)).max()
    assert float(worst) <= 1.0, float(worst)
    again = w.w4a16_gated(x, wt.packed, F, G, act=act)
    assert torch.equal(h.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("M,K,F,dtype,G,act", [c for c in GATED if c[2] < 6656])
def test_gated_grad(w, M, K, F, dtype, G, act):
    print(f"gated_grad M={M} K={K} F={F} {dtype} G={G} {act}", flush=True)
    wt = weight(w, K, 2 * F, dtype, G)
    x, x64 = normal(M * 7 + F, (M, K), dtype)
    dh, dh64 = normal(M + F, (M, F), dtype)
    dx = w.w4a16_gated_grad(x, dh, wt.packed, F, G, act=act)
    torch.cuda.synchronize()
    rows_within(dx, tu.gated_grad(wt.dev64, F, x64, dh64, act), 2 * BF + ULP[dtype], "dx")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_grad_against_differences(w, act):
    M, K, F = 6, 256, 40
    wt = weight(w, K, 2 * F, "bf16", 128)
    x, x64 = normal(1, (M, K), "bf16")
    dh, dh64 = normal(2, (M, F), "bf16")
    dx = w.w4a16_gated_grad(x, dh, wt.packed, F, 128, act=act).double()
    d = normal(3, (M, K), "bf16")[1]
    step = 1e-4
    f = lambda v: (tu.gated(wt.dev64, F, v, act) * dh64).sum(1)  # noqa: E731
    diff = (f(x64 + step * d) - f(x64 - step * d)) / (2 * step)
    # the directional derivative of a row: 3 bf16 roundings of a K-term sum, in the norm
    assert ((dx * d).sum(1) - diff).abs().max() <= 3 * BF * float((dx.norm(dim=1) * d.norm(dim=1)).max())


def test_gated_large_gates(w):
    # gates far out: the activations' limits, no infinity times zero
    K, F = 128, 16
    wt = weight(w, K, 2 * F, "bf16", 128)
    x = torch.full((4, K), 0.0, dtype=torch.bfloat16, device=DEV)
    x[0] = 1e4
    x[1] = -1e4
    x[2, ::2] = 1e30
    for act in ("silu", "gelu", "gelu_tanh"):
        h = w.w4a16_gated(x, wt.packed, F, 128, act=act)
        g, u = x.double() @ wt.dev64[:, :F], x.double() @ wt.dev64[:, F:]
        ref = torch.where(g < 0, torch.zeros_like(g), g) * u
        fine = ref.abs() < 3e38
        assert torch.isfinite(h[:2].float()).all() and not torch.isnan(h.float()).any()
        assert ((h.double() - ref).abs()[fine] <= 2 * ULP["bf16"] * ref.abs()[fine] + 1e-2).all()
        dx = w.w4a16_gated_grad(x[:2].contiguous(), torch.ones((2, F), dtype=torch.bfloat16, device=DEV), wt.packed, F, 128,
                                act=act)
        assert torch.isfinite(dx.float()).all()


# ------------------------------------------------------------------ losses

def check_loss(out, ref, x64, K, tau, dtype, dx_tol):
    value, lse, dx, _ = ref
    eps = logit_eps(x64, K) / tau
    assert ((out[1].double() - lse).abs() <= eps + 2.0 ** -20 * lse.abs()).all()
    assert ((out[0].double() - value).abs() <= tau * tau * 2 * eps + 2.0 ** -20 * (value.abs() + tau * tau * lse.abs())).all()
    if len(out) == 3:
        rows_within(out[2], dx, dx_tol, "dx")


LOSS = [
    (1, 128, 8, "bf16", 128), (1, 2048, 4096, "bf16", 128), (3, 256, 24, "fp16", 64), (16, 512, 1000, "bf16", 32),
    (17, 384, 136, "fp16", -1), (40, 1024, 5000, "bf16", 128), (64, 256, 2056, "fp16", 128), (65, 512, 264, "bf16", 64),
    (130, 2048, 3000, "bf16", 128), (300, 256, 9000, "fp16", 256),
]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M,K,V,dtype,G", LOSS)
def test_cross_entropy(w, M, K, V, dtype, G, grad):
    print(f"cross_entropy M={M} K={K} V={V} {dtype} G={G} grad={grad}", flush=True)
    wt = weight(w, K, V, dtype, G)
    x, x64 = normal(M + V, (M, K), dtype)
    rng = np.random.default_rng(V)
    labels = rng.integers(0, V, size=M).astype(np.int32)
    labels[0], labels[-1] = V - 1, 0
    if M > 4:
        labels[2], labels[3] = -100, V                 # ignored
    lab = torch.from_numpy(labels).to(DEV)
    dloss = torch.from_numpy(rng.uniform(0.5, 2.0, M).astype(np.float32)).to(DEV)
    out = w.w4a16_cross_entropy(x, lab, wt.packed, V, G, grad=grad, dloss=dloss if grad else None)
    torch.cuda.synchronize()
    p = ((lab >= 0) & (lab < V)).double()[:, None]
    ref = tu.loss(wt.dev64, x64, lab[:, None].long(), p, 1.0, dloss.double())
    check_loss(out, ref, x64, K, 1.0, dtype, 2 * BF + ULP[dtype])
    again = w.w4a16_cross_entropy(x, lab, wt.packed, V, G, grad=grad, dloss=dloss if grad else None)
    for a, b in zip(out, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if M > 4:
        assert out[0][2] == 0 and out[0][3] == 0
        if grad:
            assert (out[2][2:4] == 0).all()


@pytest.mark.parametrize("M,K,V,dtype,G,T,tau", [
    (1, 128, 8, "bf16", 128, 1, 1.0), (5, 256, 1000, "fp16", 64, 7, 2.0), (16, 512, 520, "bf16", -1, 64, 1.0),
    (33, 256, 4104, "bf16", 128, 20, 3.5), (70, 384, 2000, "fp16", 32, 128, 1.0), (140, 1024, 6000, "bf16", 128, 256, 2.0),
])
def test_distill(w, M, K, V, dtype, G, T, tau):
    print(f"distill M={M} K={K} V={V} {dtype} G={G} T={T}", flush=True)
    wt = weight(w, K, V, dtype, G)
    x, x64 = normal(M * 3 + V, (M, K), dtype)
    rng = np.random.default_rng(T)
    ids = rng.integers(0, V, size=(M, T)).astype(np.int32)        # duplicates where T is large
    t = (3 * rng.standard_normal((M, T))).astype(np.float32)
    if M > 8:
        ids[1] = -1                                               # nothing left
        ids[2, 1:] = V                                            # one entry
        t[3, T // 2:] = -np.inf
        t[4] = -np.inf                                            # nothing left
        ids[5] = 7                                                # one id, every weight
        t[6] = 60.0 * np.sign(t[6])                               # nearly one-hot
    ids, t = torch.from_numpy(ids).to(DEV), torch.from_numpy(t).to(DEV)
    dloss = torch.from_numpy(rng.uniform(0.5, 2.0, M).astype(np.float32)).to(DEV)
    out = w.w4a16_distill(x, ids, t, wt.packed, V, G, temperature=tau, grad=True, dloss=dloss)
    torch.cuda.synchronize()
    p = tu.teacher(ids, t, V, tau)
    ref = tu.loss(wt.dev64, x64, ids.long(), p, tau, dloss.double())
    check_loss(out, ref, x64, K, tau, dtype, 2 * BF + ULP[dtype])
    if M > 8:
        assert out[0][1] == 0 and out[0][4] == 0 and (out[2][[1, 4]] == 0).all()
    plain = w.w4a16_distill(x, ids, t, wt.packed, V, G, temperature=tau)
    assert torch.equal(plain[0], out[0]) and torch.equal(plain[1], out[1])


def test_distill_of_one_entry_is_cross_entropy(w):
    M, K, V = 20, 256, 1000
    wt = weight(w, K, V, "bf16", 128)
    x, _ = normal(9, (M, K), "bf16")
    ids = torch.arange(M, dtype=torch.int32, device=DEV) * 49
    ce = w.w4a16_cross_entropy(x, ids, wt.packed, V, 128, grad=True)
    di = w.w4a16_distill(x, ids[:, None].contiguous(), torch.zeros((M, 1), device=DEV), wt.packed, V, 128, grad=True)
    for a, b in zip(ce, di):
        assert torch.equal(a, b)


def test_loss_ignored_rows_may_hold_anything(w):
    M, K, V = 24, 256, 1000
    wt = weight(w, K, V, "bf16", 128)
    x, x64 = normal(10, (M, K), "bf16")
    lab = torch.arange(M, dtype=torch.int32, device=DEV) * 40
    lab[[3, 17]] = -100
    clean = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True)
    dirty = x.clone()
    dirty[3] = float("nan")
    dirty[17] = float("inf")
    out = w.w4a16_cross_entropy(dirty, lab, wt.packed, V, 128, grad=True)
    assert (out[0][[3, 17]] == 0).all() and (out[2][[3, 17]] == 0).all()
    keep = [m for m in range(M) if m not in (3, 17)]
    assert torch.equal(out[0][keep], clean[0][keep]) and torch.equal(out[2][keep], clean[2][keep])


def test_loss_far_logits(w):
    # logits of several thousand: the maximum is taken off before the exponential
    M, K, V = 8, 256, 1000
    wt = weight(w, K, V, "bf16", 128)
    x, x64 = normal(11, (M, K), "bf16", scale=1000.0)
    lab = torch.arange(M, dtype=torch.int32, device=DEV)
    out = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True)
    ref = tu.loss(wt.dev64, x64, lab[:, None].long(), torch.ones((M, 1), dtype=torch.float64, device=DEV), 1.0,
                  torch.ones(M, dtype=torch.float64, device=DEV))
    eps = logit_eps(x64, K)
    assert ((out[0].double() - ref[0]).abs() <= 2 * eps + 2.0 ** -20 * ref[1].abs()).all()
    assert torch.isfinite(out[2].float()).all()


def test_cross_entropy_confident_row(w):
    # x along the label's own column: q_label near 1, the gradient is a small difference
    K, V = 512, 2000
    wt = weight(w, K, V, "bf16", 128)
    cols = torch.tensor([5, 700, 1999], device=DEV)
    x64 = wt.dev64[:, cols].t() * 3.0
    x = x64.to(torch.bfloat16).contiguous()
    lab = cols.to(torch.int32)
    out = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True)
    ref = tu.loss(wt.dev64, x.double(), lab[:, None].long(), torch.ones((3, 1), dtype=torch.float64, device=DEV), 1.0,
                  torch.ones(3, dtype=torch.float64, device=DEV))
    # q - 1 in fp32 off by 2^-24 and the logits' error: relative to 1 - q
    rest = 1 - torch.exp(-ref[0])
    extra = ((logit_eps(x.double(), K) + 2.0 ** -22) * 2 / rest).max()
    rows_within(out[2], ref[2], 3 * BF + float(extra), "dx")


def test_cross_entropy_against_differences(w):
    # x on a grid of 1/16 and a step of 1/64: both sides exact in bf16. The central
    # difference's own error is step^2 / 6 of the third derivative along d, at most
    # max |z'|^3 of the direction's logits
    M, K, V = 12, 128, 200
    wt = weight(w, K, V, "bf16", 128)
    rng = np.random.default_rng(4)
    x64 = torch.from_numpy(rng.integers(-16, 17, (M, K)) / 16.0).to(DEV)
    d64 = torch.from_numpy(rng.integers(-1, 2, (M, K)).astype(np.float64)).to(DEV)
    lab = torch.from_numpy(rng.integers(0, V, M).astype(np.int32)).to(DEV)
    step = 1.0 / 64
    f = lambda v: w.w4a16_cross_entropy(v.to(torch.bfloat16), lab, wt.packed, V, 128)[0].double()  # noqa: E731
    diff = (f(x64 + step * d64) - f(x64 - step * d64)) / (2 * step)
    dx = w.w4a16_cross_entropy(x64.to(torch.bfloat16), lab, wt.packed, V, 128, grad=True)[2].double()
    zd = (d64 @ wt.dev64).abs().max(dim=1).values
    eps = logit_eps(x64 + step, K)
    tol = step ** 2 / 6 * 2 * zd ** 3 + 2 * eps / step + 3 * BF * dx.norm(dim=1) * d64.norm(dim=1) / np.sqrt(K) * 3
    assert (((dx * d64).sum(1) - diff).abs() <= tol).all()


# ------------------------------------------------------------------ pieces, streams, graphs

def test_pieces_of_the_vocabulary_and_rows(w):
    # more rows than one pass takes, and a head of several pieces
    M, K, V = 4096 + 130, 128, 40000
    wt = weight(w, K, V, "bf16", 128)
    x, x64 = normal(12, (M, K), "bf16")
    lab = torch.from_numpy(np.random.default_rng(1).integers(0, V, M).astype(np.int32)).to(DEV)
    out = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True)
    one = torch.ones((M, 1), dtype=torch.float64, device=DEV)
    ref = tu.loss(wt.dev64, x64, lab[:, None].long(), one, 1.0, one[:, 0])
    check_loss(out, ref, x64, K, 1.0, "bf16", 3 * BF)


def test_gated_grad_more_rows_than_a_pass(w):
    M, K, F = 8192 + 70, 128, 40
    wt = weight(w, K, 2 * F, "bf16", 128)
    x, x64 = normal(13, (M, K), "bf16")
    dh, dh64 = normal(14, (M, F), "bf16")
    dx = w.w4a16_gated_grad(x, dh, wt.packed, F, 128)
    rows_within(dx, tu.gated_grad(wt.dev64, F, x64, dh64, "silu"), 3 * BF, "dx")


def test_one_workspace_serves_every_entry(w):
    # a K-split GEMM, the losses and the gradients on one zeroed workspace, in turn
    K, V, M = 6656, 512, 16
    wt = weight(w, K, V, "bf16", 128)
    x, x64 = normal(15, (M, K), "bf16")
    need = max(w.w4a16_workspace_bytes(M, K, V, 128), w.w4a16_cross_entropy_workspace_bytes(M, K, V, 128, True),
               w.w4a16_gated_workspace_bytes(M, K, V // 2, 128, True), w.w4a16_gemm_grad_workspace_bytes(M, K, V, 128))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    lab = torch.arange(M, dtype=torch.int32, device=DEV)
    first = None
    for _ in range(3):
        y = w.w4a16_gemm(x, wt.packed, V, 128, workspace=ws)
        ce = w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True, workspace=ws)
        h = w.w4a16_gated(x, wt.packed, V // 2, 128, workspace=ws)
        dx = w.w4a16_gated_grad(x, h, wt.packed, V // 2, 128, workspace=ws)
        dy = w.w4a16_gemm_grad(y, wt.packed, K, 128, workspace=ws)
        assert (ws[:512] == 0).all()
        now = [t.clone() for t in (y, *ce, h, dx, dy)]
        if first is not None:
            for a, b in zip(first, now):
                assert torch.equal(a, b)
        first = now
    assert norm_err(first[0], x64 @ wt.dev64) <= 2 * BF


def test_side_stream_and_graph(w):
    M, K, V, F = 48, 256, 2000, 1000
    wt = weight(w, K, V, "bf16", 128)
    lab = torch.arange(M, dtype=torch.int32, device=DEV) * 3
    xs = [normal(20 + i, (M, K), "bf16")[0] for i in range(3)]
    eager = [(w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True), w.w4a16_gated(x, wt.packed, F, 128),
              w.w4a16_gated_grad(x, w.w4a16_gated(x, wt.packed, F, 128), wt.packed, F, 128)) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = w.w4a16_cross_entropy(xs[0], lab, wt.packed, V, 128, grad=True)
    side.synchronize()
    for a, b in zip(got, eager[0][0]):
        assert torch.equal(a, b)
    x = xs[0].clone()
    need = max(w.w4a16_cross_entropy_workspace_bytes(M, K, V, 128, True), w.w4a16_gated_workspace_bytes(M, K, F, 128, True))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    h, dx, gx = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((M, F), (M, K), (M, K)))
    loss, lse = (torch.empty(M, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.w4a16_cross_entropy(x, lab, wt.packed, V, 128, grad=True, loss=loss, lse=lse, dx=dx, workspace=ws)
        w.w4a16_gated(x, wt.packed, F, 128, h=h, workspace=ws)
        w.w4a16_gated_grad(x, h, wt.packed, F, 128, dx=gx, workspace=ws)
    for i in (0, 1, 2, 1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        (l0, e0, d0), h0, g0 = eager[i]
        assert torch.equal(loss, l0) and torch.equal(lse, e0) and torch.equal(dx, d0)
        assert torch.equal(h, h0) and torch.equal(gx, g0)
        w.w4a16_gated(xs[2], wt.packed, F, 128)       # the program's own work between replays


def test_outputs_written_in_full_and_nothing_past_them(w):
    M, K, F = 19, 256, 40
    wt = weight(w, K, 2 * F, "bf16", 128)
    x, _ = normal(30, (M, K), "bf16")
    room = torch.full((M * F + 64,), -7.0, dtype=torch.bfloat16, device=DEV)
    h = room[:M * F].view(M, F)
    w.w4a16_gated(x, wt.packed, F, 128, h=h)
    assert (room[M * F:] == -7.0).all() and not (h == -7.0).all(dim=0).any()
    room = torch.full((M * K + 64,), -7.0, dtype=torch.bfloat16, device=DEV)
    w.w4a16_gated_grad(x, h, wt.packed, F, 128, dx=room[:M * K].view(M, K))
    assert (room[M * K:] == -7.0).all()
    room = torch.full((M * K + 64,), -7.0, dtype=torch.bfloat16, device=DEV)
    w.w4a16_cross_entropy(x, torch.zeros(M, dtype=torch.int32, device=DEV), wt.packed, 2 * F, 128, grad=True,
                          dx=room[:M * K].view(M, K))
    assert (room[M * K:] == -7.0).all()


def test_no_rows(w):
    K, F = 256, 40
    wt = weight(w, K, 2 * F, "bf16", 128)
    x = torch.empty((0, K), dtype=torch.bfloat16, device=DEV)
    assert w.w4a16_gated(x, wt.packed, F, 128).shape == (0, F)
    assert w.w4a16_gated_grad(x, torch.empty((0, F), dtype=torch.bfloat16, device=DEV), wt.packed, F, 128).shape == (0, K)
    assert w.w4a16_gemm_grad(torch.empty((0, 2 * F), dtype=torch.bfloat16, device=DEV), wt.packed, K, 128).shape == (0, K)
    out = w.w4a16_cross_entropy(x, torch.empty(0, dtype=torch.int32, device=DEV), wt.packed, 2 * F, 128, grad=True)
    assert out[0].shape == (0,) and out[2].shape == (0, K)
