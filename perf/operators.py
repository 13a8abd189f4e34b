"""The operators that train through, and score with, frozen int4 weights: a gated
feed-forward block, the softmax cross entropy and the distillation loss over a packed
output head, and the product's gradient. Cases, inputs, plain forms and exact values.

Every case holds one packed weight in the library's tile layout (version 2), as
`load_packed` would bring it in: W[k, n] = (q[k, n] - z[k div G, n]) * s[k div G, n].
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decoded token through the gate_up layer: bound by latency and weight bytes
        {"name": "gated_token", "op": "gated", "dtype": "bf16", "M": 1, "K": 2048, "N": 6656, "G": 128, "act": "silu"},
        # a batch of decoded sequences, odd in number
        {"name": "gated_batch13", "op": "gated", "dtype": "fp16", "M": 13, "K": 2048, "N": 6656, "G": 128, "act": "gelu_tanh"},
        # a prompt of 512 tokens
        {"name": "gated_prompt", "op": "gated", "dtype": "bf16", "M": 512, "K": 2048, "N": 6656, "G": 128, "act": "silu"},
        # backward of the block: a training batch of 4096 tokens
        {"name": "gated_grad_train", "op": "gated_grad", "dtype": "bf16", "M": 4096, "K": 2048, "N": 6656, "G": 128, "act": "silu"},
        # backward of the block on a short ragged batch, finer groups, a width that ends in half a column block
        {"name": "gated_grad_ragged", "op": "gated_grad", "dtype": "fp16", "M": 333, "K": 1024, "N": 2728, "G": 64, "act": "gelu"},
        # backward of the down projection: a training batch
        {"name": "gemm_grad_down", "op": "gemm_grad", "dtype": "bf16", "M": 4096, "K": 6656, "N": 2048, "G": 128},
        # backward of a projection for one short sequence
        {"name": "gemm_grad_short", "op": "gemm_grad", "dtype": "fp16", "M": 77, "K": 2048, "N": 2056, "G": 128},
        # log-probability of one token under the full head (scoring while serving)
        {"name": "ce_token", "op": "ce", "dtype": "bf16", "M": 1, "K": 2048, "N": 131072, "G": 128, "grad": False},
        # scoring a short text over a smaller vocabulary, some positions not scored
        {"name": "ce_text", "op": "ce", "dtype": "fp16", "M": 333, "K": 1024, "N": 32008, "G": 64, "grad": False},
        # loss and gradient of a training batch over the full head
        {"name": "ce_train", "op": "ce", "dtype": "bf16", "M": 4096, "K": 2048, "N": 131072, "G": 128, "grad": True},
        # distillation step: teacher's top 64 of the full vocabulary
        {"name": "distill_train", "op": "distill", "dtype": "bf16", "M": 1024, "K": 2048, "N": 131072, "G": 128, "T": 64, "tau": 2.0, "grad": True},
        # distillation on a small ragged batch, short lists
        {"name": "distill_ragged", "op": "distill", "dtype": "fp16", "M": 65, "K": 1024, "N": 32008, "G": -1, "T": 20, "tau": 1.0, "grad": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "gemm_grad", "ce", "distill"])
    G = rng.choice([128, 128, 128, 256, 64, 32, -1])
    K = 256 * _log_int(rng, 1, 16)
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "M": _log_int(rng, 1, 4096), "K": K, "G": G}
    if op in ("gated", "gated_grad"):
        c["N"] = 8 * _log_int(rng, 32, 1024)
        c["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    elif op == "gemm_grad":
        c["N"] = 8 * _log_int(rng, 32, 1024)
    else:
        c["N"] = 8 * _log_int(rng, 125, 16384)
        c["K"] = min(K, 2048)
        c["grad"] = rng.random() < 0.6
        if op == "distill":
            c["T"] = _log_int(rng, 1, 128)
            c["tau"] = rng.choice([1.0, 1.0, 2.0, 3.5])
    return c


def _columns(case):
    return 2 * case["N"] if case["op"] in ("gated", "gated_grad") else case["N"]


def _layout(case):
    """(K, columns, columns rounded up to whole blocks, rows of a metadata unit, words per column)"""
    K, N = case["K"], _columns(case)
    G = K if case["G"] == -1 else case["G"]
    unit = min(G, 128)
    return K, N, (N + 15) // 16 * 16, G, unit, (K // unit + 3) // 4 * 4


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 17)
    dt = _DT[case["dtype"]]
    K, N, Np, G, unit, words = _layout(case)
    M = case["M"]

    # the packed weight: uniform codes and zero points, scales uniform on [0.005, 0.02);
    # the padding of a last half block is zero
    codes = torch.randint(-2 ** 31, 2 ** 31, (Np // 16, K // 128, 4, 16, 4), generator=gen, device=dev, dtype=torch.int32)
    if Np != N:
        codes[-1, :, :, 8:, :] = 0
    scale = (torch.rand((N, K // G), generator=gen, device=dev) * 0.015 + 0.005).to(dt)
    zero = torch.randint(0, 16, (N, K // G), generator=gen, device=dev, dtype=torch.int32)
    word = (scale.view(torch.int16).to(torch.int32) & 0xFFFF) | (zero << 16)
    meta = torch.zeros((Np, words), dtype=torch.int32, device=dev)
    meta[:N, :K // unit] = word.repeat_interleave(G // unit, dim=1)
    packed = torch.cat([codes.view(torch.uint8).reshape(-1), meta.view(torch.uint8).reshape(-1)])

    s = {"case": case, "packed": packed}
    # fp16 training scales its loss so that small gradients stay in range
    lift = 1024.0 if case["dtype"] == "fp16" else 1.0
    if case["op"] == "gemm_grad":
        s["dy"] = (torch.randn((M, N), generator=gen, device=dev) * (lift * 1e-3)).to(dt)
        return s
    s["x"] = torch.randn((M, K), generator=gen, device=dev).to(dt)
    if case["op"] == "gated_grad":
        s["dh"] = (torch.randn((M, case["N"]), generator=gen, device=dev) * (lift * 1e-3)).to(dt)
    if case["op"] in ("ce", "distill"):
        s["dloss"] = torch.full((M,), lift / M, device=dev)
    if case["op"] == "ce":
        s["labels"] = torch.randint(0, N, (M,), generator=gen, device=dev, dtype=torch.int32)
        if M >= 16:   # positions without a label: prompts, padding
            s["labels"][torch.rand((M,), generator=gen, device=dev) < 0.1] = -100
    if case["op"] == "distill":
        T = case["T"]
        # distinct ids per row: a random start and a random odd stride over the vocabulary
        start = torch.randint(0, N, (M, 1), generator=gen, device=dev)
        stride = 1 + torch.randint(0, max(1, N // (2 * T)), (M, 1), generator=gen, device=dev)
        ids = ((start + stride * torch.arange(T, device=dev)) % N).to(torch.int32)
        logits = (3.0 * torch.randn((M, T), generator=gen, device=dev)).sort(dim=1, descending=True).values
        if T >= 8:    # some lists are shorter: padded with id -1
            short = torch.rand((M,), generator=gen, device=dev) < 0.1
            ids[short, T // 2:] = -1
        s["top_ids"], s["top_logits"] = ids, logits
    return s


# ------------------------------------------------------------------ plain forms

def _plain_weight(s):
    """The packed buffer -> W [K, columns] in 32 bits."""
    case = s["case"]
    K, N, Np, G, unit, words = _layout(case)
    nb = K * Np // 2
    # block [column block, row block, lane quarter h, column c, word i]: rows 32 i + 8 h + e
    w = s["packed"][:nb].view(torch.int32).view(Np // 16, K // 128, 4, 16, 4)
    q = torch.stack([(w >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15 for e in range(8)], dim=-1)
    q = q.permute(1, 4, 2, 5, 0, 3).reshape(K, Np)[:, :N].float()
    meta = s["packed"][nb:].view(torch.int32).view(Np, words)[:N, :K // unit]
    z = ((meta >> 16) & 15).t().float()
    sc = (meta & 0xFFFF).to(torch.int16).view(_DT[case["dtype"]]).t().float()
    q = q.view(K // unit, unit, N)
    return ((q - z[:, None, :]) * sc[:, None, :]).view(K, N)


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(name, g):
    if name == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return e * (1.0 + g * (1.0 - e))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain_gated(s):
    F = s["case"]["N"]
    y = s["x"].float() @ _plain_weight(s)
    return (_act(s["case"]["act"], y[:, :F]) * y[:, F:]).to(s["x"].dtype)


def _plain_gated_grad(s):
    F, act = s["case"]["N"], s["case"]["act"]
    W = _plain_weight(s)
    y = s["x"].float() @ W
    g, u, dh = y[:, :F], y[:, F:], s["dh"].float()
    d = torch.cat([dh * u * _act_slope(act, g), dh * _act(act, g)], dim=1)
    return (d @ W.t()).to(s["x"].dtype)


def _plain_gemm_grad(s):
    return (s["dy"].float() @ _plain_weight(s).t()).to(s["dy"].dtype)


def _plain_targets(s):
    """(ids, weights) of each row's targets; a row without a valid one has weights of zero."""
    case = s["case"]
    if case["op"] == "ce":
        ids = s["labels"].long()[:, None]
        ok = (ids >= 0) & (ids < case["N"])
        return ids.clamp(0, case["N"] - 1), ok.float()
    ids = s["top_ids"].long()
    ok = (ids >= 0) & (ids < case["N"])
    t = torch.where(ok, s["top_logits"] / case["tau"], torch.full_like(s["top_logits"], -math.inf))
    top = t.max(dim=1, keepdim=True).values
    e = torch.exp(t - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(dim=1, keepdim=True)
    return ids.clamp(0, case["N"] - 1), e / torch.where(total == 0, torch.ones_like(total), total)


def _plain_loss(s):
    case = s["case"]
    tau = case.get("tau", 1.0)
    W = _plain_weight(s)
    z = (s["x"].float() @ W) / tau
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    lse = top + torch.log(total)
    ids, p = _plain_targets(s)
    some = (p.sum(dim=1) > 0).float()
    logp = torch.where(p > 0, torch.log(p), torch.zeros_like(p))
    loss = tau * tau * (p * (logp - z.gather(1, ids) + lse)).sum(dim=1)
    if not case["grad"]:
        return loss, lse[:, 0]
    d = (e / total) * some[:, None]
    d.scatter_add_(1, ids, -p)
    dx = ((s["dloss"] * tau)[:, None] * (d @ W.t())).to(s["x"].dtype)
    return loss, lse[:, 0], dx


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "gated":
            return _plain_gated(state)
        if op == "gated_grad":
            return _plain_gated_grad(state)
        if op == "gemm_grad":
            return _plain_gemm_grad(state)
        return _plain_loss(state)
    import w4a16_int4_weight_amd as w
    if op == "gated":
        return w.w4a16_gated(state["x"], state["packed"], case["N"], case["G"], act=case["act"])
    if op == "gated_grad":
        return w.w4a16_gated_grad(state["x"], state["dh"], state["packed"], case["N"], case["G"], act=case["act"])
    if op == "gemm_grad":
        return w.w4a16_gemm_grad(state["dy"], state["packed"], case["K"], case["G"])
    if op == "ce":
        return w.w4a16_cross_entropy(state["x"], state["labels"], state["packed"], case["N"], case["G"],
                                     grad=case["grad"], dloss=state["dloss"] if case["grad"] else None)
    return w.w4a16_distill(state["x"], state["top_ids"], state["top_logits"], state["packed"], case["N"], case["G"],
                           temperature=case["tau"], grad=case["grad"], dloss=state["dloss"] if case["grad"] else None)


def work(case):
    op, M = case["op"], case["M"]
    K, N, Np, G, unit, words = _layout(case)
    # codes, and one 16-bit scale and one 4-bit zero point per column and group
    weight = K * N / 2 + (K // G) * N * 2.5
    product = 2.0 * M * K * N
    if op == "gated":
        return {"bytes": weight + 2 * M * (K + case["N"]), "flops": product}
    if op == "gated_grad":
        return {"bytes": weight + 2 * M * (2 * K + case["N"]), "flops": 2 * product}
    if op == "gemm_grad":
        return {"bytes": weight + 2 * M * (K + N), "flops": product}
    rows = 2 * M * K + 8 * M + (4 * M if op == "ce" else 8 * M * case["T"])
    if case["grad"]:
        return {"bytes": weight + rows + 4 * M + 2 * M * K, "flops": 2 * product}
    return {"bytes": weight + rows, "flops": product}


# ------------------------------------------------------------------ 64 bits, from the definition

def _exact_weight(s):
    """W by address: element (k, n) of the layout, one lookup each, in 64 bits."""
    case = s["case"]
    K, N, Np, G, unit, words = _layout(case)
    dev = s["packed"].device
    W = torch.empty((N, K), dtype=torch.float64, device=dev)
    k = torch.arange(K, device=dev)
    row, sub = k // 128, k % 128
    within = ((sub % 32) // 8) * 256 + (sub // 32) * 4          # byte of the word in its 1 KiB block, column 0
    pos = k % 8
    nibble = torch.where(pos % 2 == 0, pos // 2, 4 + pos // 2)
    nbytes = K * Np // 2
    for n0 in range(0, N, 16384):
        n = torch.arange(n0, min(n0 + 16384, N), device=dev)[:, None]
        byte = ((n // 16) * (K // 128) + row) * 1024 + within + (n % 16) * 16 + nibble // 2
        q = (s["packed"][byte] >> (4 * (nibble % 2)).to(torch.uint8)) & 15
        m = nbytes + 4 * (n * words + k // unit)
        z = s["packed"][m + 2] & 15
        bits = s["packed"][m].to(torch.int32) | (s["packed"][m + 1].to(torch.int32) << 8)
        sc = bits.to(torch.int16).view(_DT[case["dtype"]]).double()
        W[n0:n0 + 16384] = (q.double() - z.double()) * sc
    return W


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], _DT[case["dtype"]]
    Wt = _exact_weight(s)                                      # [columns, K]
    if op == "gemm_grad":
        return s["dy"].double() @ Wt
    x = s["x"].double()
    F = case["N"]
    if op in ("gated", "gated_grad"):
        g, u = x @ Wt[:F].t(), x @ Wt[F:].t()
        c = math.sqrt(2.0 / math.pi)
        if case["act"] == "silu":
            e = torch.sigmoid(g)
            a, da = g * e, e + g * e * (1 - e)
        elif case["act"] == "gelu":
            e = 0.5 * torch.erfc(-g * math.sqrt(0.5))
            a, da = g * e, e + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        else:
            e = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
            a, da = g * e, e + 2 * g * e * (1 - e) * c * (1 + 0.134145 * g * g)
        if op == "gated":
            return a * u
        dh = s["dh"].double()
        return (dh * u * da) @ Wt[:F] + (dh * a) @ Wt[F:]
    V, M = case["N"], case["M"]
    tau = case.get("tau", 1.0)
    logq = torch.log_softmax((x @ Wt.t()) / tau, dim=1)
    if op == "ce":
        ids, t = s["labels"].long()[:, None], torch.zeros((M, 1), dtype=torch.float64, device=x.device)
    else:
        ids, t = s["top_ids"].long(), s["top_logits"].double() / tau
    ok = (ids >= 0) & (ids < V)
    ids = torch.where(ok, ids, torch.zeros_like(ids))
    p = torch.softmax(torch.where(ok, t, torch.full_like(t, -math.inf)), dim=1)
    p = torch.where(ok, p, torch.zeros_like(p))                # rows without a target: softmax gives NaN
    target = torch.zeros_like(logq).scatter_add_(1, ids, p)
    loss = tau ** 2 * (torch.special.xlogy(p, p).sum(1) - (target * logq).sum(1))
    lse = (x @ Wt[:1].t())[:, 0] / tau - logq[:, 0]
    if not case["grad"]:
        return loss, lse
    q = torch.exp(logq) * ok.any(dim=1, keepdim=True)
    dx = (tau * s["dloss"].double())[:, None] * ((q - target) @ Wt)
    return loss, lse, dx
