"""The operators of a decoding step over a mixture of int4 experts: the router's choice of
experts, the experts' layer on packed weights, and the draw of the next token from the
head's logits. Cases, inputs, plain forms and exact values.

Packed weights are in the library's tile layout (version 2), one expert after another, as
`load_packed` would bring each in: W[k, n] = (q[k, n] - z[k div G, n]) * s[k div G, n].
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the router of one decoded token
        {"name": "route_token", "op": "route", "dtype": "bf16", "M": 1, "K": 2048, "E": 64, "T": 8, "score": "softmax", "normalize": True, "bias": False, "scale": 1.0},
        # the router of a prompt: gates of their own, a balancing bias that enters the choice alone
        {"name": "route_prompt", "op": "route", "dtype": "bf16", "M": 512, "K": 2048, "E": 128, "T": 8, "score": "sigmoid", "normalize": True, "bias": True, "scale": 2.5},
        # experts of one decoded token: bound by latency and the routed experts' bytes
        {"name": "moe_token", "op": "moe", "dtype": "bf16", "M": 1, "K": 2048, "F": 1024, "E": 64, "T": 8, "G": 128, "act": "silu", "residual": True},
        # an odd number of sequences, finer groups, a narrow layer, some tokens dropped
        {"name": "moe_batch13", "op": "moe", "dtype": "fp16", "M": 13, "K": 1024, "F": 640, "E": 32, "T": 4, "G": 64, "act": "gelu_tanh", "residual": False},
        # a short prompt, more rows than a decoding batch: experts meet 2 to 20 rows each
        {"name": "moe_prompt77", "op": "moe", "dtype": "bf16", "M": 77, "K": 2048, "F": 1024, "E": 64, "T": 8, "G": 128, "act": "silu", "residual": True},
        # the whole layer of a decoding batch
        {"name": "layer_batch16", "op": "layer", "dtype": "bf16", "M": 16, "K": 2048, "F": 1024, "E": 64, "T": 8, "G": 128, "act": "silu", "residual": True, "score": "softmax", "normalize": True, "bias": False, "scale": 1.0},
        # the whole layer of a prompt
        {"name": "layer_prompt", "op": "layer", "dtype": "bf16", "M": 512, "K": 2048, "F": 1024, "E": 64, "T": 8, "G": 128, "act": "silu", "residual": True, "score": "softmax", "normalize": True, "bias": False, "scale": 1.0},
        # one sequence's next token from the whole vocabulary: nucleus sampling
        {"name": "sample_token", "op": "sample", "dtype": "bf16", "M": 1, "V": 131072, "pad": 0, "t": 0.8, "k": 0, "p": 0.95, "min_p": 0.0, "rows": False},
        # an odd batch over a smaller, padded vocabulary, logits processed in 32 bits, every row with its own settings
        {"name": "sample_rows13", "op": "sample", "dtype": "fp32", "M": 13, "V": 32003, "pad": 5, "t": 1.0, "k": 40, "p": 0.9, "min_p": 0.02, "rows": True},
        # a serving batch: the usual top-k and top-p
        {"name": "sample_batch64", "op": "sample", "dtype": "bf16", "M": 64, "V": 131072, "pad": 0, "t": 0.7, "k": 50, "p": 0.9, "min_p": 0.0, "rows": False},
        # many rollouts at once, drawn from the model's own distribution
        {"name": "sample_rollouts", "op": "sample", "dtype": "fp16", "M": 256, "V": 131072, "pad": 0, "t": 1.0, "k": 0, "p": 1.0, "min_p": 0.0, "rows": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "layer", "sample", "sample"])
    if op == "sample":
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "M": _log_int(rng, 1, 128), "V": _log_int(rng, 500, 131072),
                "pad": rng.choice([0, 0, 3, 8]), "t": rng.choice([0.0, 0.6, 1.0, 1.0, 1.4]), "k": rng.choice([0, 0, 1, 20, 100, 1000]),
                "p": rng.choice([1.0, 1.0, 0.5, 0.9, 0.99]), "min_p": rng.choice([0.0, 0.0, 0.05]), "rows": rng.random() < 0.4}
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "M": _log_int(rng, 1, 384), "K": 256 * _log_int(rng, 1, 8),
         "E": rng.choice([4, 8, 16, 24, 60, 64])}
    c["T"] = rng.randint(1, min(8, c["E"]))
    if op != "route":
        c.update(F=128 * rng.randint(1, 8), G=rng.choice([128, 128, 128, 64, 32, -1]), act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                 residual=rng.random() < 0.7)
    if op != "moe":
        c.update(score=rng.choice(["softmax", "softmax", "sigmoid"]), normalize=rng.random() < 0.7, bias=rng.random() < 0.3,
                 scale=rng.choice([1.0, 1.0, 2.5]))
    return c


def _sizes(K, N, G):
    """(columns rounded up to whole blocks, rows of a group, rows of a metadata unit, words per column)"""
    G = K if G == -1 else G
    unit = min(G, 128)
    return (N + 15) // 16 * 16, G, unit, (K // unit + 3) // 4 * 4


def _experts(gen, E, K, N, G, dt):
    """E packed weights: uniform codes and zero points, scales uniform on [0.005, 0.02)."""
    dev = gen.device
    Np, G, unit, words = _sizes(K, N, G)
    codes = torch.randint(-2 ** 31, 2 ** 31, (E, K * Np // 8), generator=gen, device=dev, dtype=torch.int32)
    scale = (torch.rand((E, N, K // G), generator=gen, device=dev) * 0.015 + 0.005).to(dt)
    zero = torch.randint(0, 16, (E, N, K // G), generator=gen, device=dev, dtype=torch.int32)
    word = (scale.view(torch.int16).to(torch.int32) & 0xFFFF) | (zero << 16)
    meta = torch.zeros((E, Np, words), dtype=torch.int32, device=dev)
    meta[:, :N, :K // unit] = word.repeat_interleave(G // unit, dim=2)
    return torch.cat([codes, meta.reshape(E, -1)], dim=1).view(torch.uint8)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 29)
    dt = _DT[case["dtype"]]
    M = case["M"]
    s = {"case": case}
    if case["op"] == "sample":
        V = case["V"]
        # a bell of unlikely tokens and a few likely ones; some rows have banned tokens
        z = 2.2 * torch.randn((M, V + case["pad"]), generator=gen, device=dev)
        likely = torch.randint(0, V, (M, 12), generator=gen, device=dev)
        z.scatter_add_(1, likely, 4.0 + 8.0 * torch.rand((M, 12), generator=gen, device=dev))
        banned = torch.rand((M, 1), generator=gen, device=dev) < 0.3
        z.masked_fill_(banned & (torch.rand(z.shape, generator=gen, device=dev) < 0.05), -math.inf)
        s["logits"] = z.to(dt)[:, :V]
        s["u"] = torch.rand((M,), generator=gen, device=dev)
        s["t"], s["k"], s["p"], s["min_p"] = case["t"], case["k"], case["p"], case["min_p"]
        if case["rows"]:           # one request's settings beside another's
            r = torch.rand((4, M), generator=gen, device=dev)
            s["t"] = torch.where(r[0] < 0.15, torch.zeros_like(r[0]), case["t"] * (0.5 + r[0]))
            s["k"] = torch.where(r[1] < 0.3, torch.zeros_like(r[1]), case["k"] * 2 * r[1]).to(torch.int32)
            s["p"] = torch.where(r[2] < 0.3, torch.ones_like(r[2]), 1 - (1 - case["p"]) * 2 * r[2])
            s["min_p"] = case["min_p"] * 2 * r[3]
        return s
    K, E, T = case["K"], case["E"], case["T"]
    s["x"] = torch.randn((M, K), generator=gen, device=dev).to(dt)
    if case["op"] != "moe":
        s["router"] = (torch.randn((E, K), generator=gen, device=dev) * (1.5 / math.sqrt(K))).to(dt)
        s["bias"] = 0.1 * torch.randn((E,), generator=gen, device=dev) if case["bias"] else None
    else:
        s["ids"] = torch.rand((M, E), generator=gen, device=dev).argsort(dim=1)[:, :T].to(torch.int32)
        s["weights"] = torch.softmax(torch.randn((M, T), generator=gen, device=dev), dim=1)
        if M >= 8:                 # entries dropped for capacity, and padding rows
            s["ids"][torch.rand((M, T), generator=gen, device=dev) < 0.05] = -1
            s["ids"][M - 1] = -1
    if case["op"] != "route":
        s["gate_up"] = _experts(gen, E, K, 2 * case["F"], case["G"], dt)
        s["down"] = _experts(gen, E, case["F"], K, case["G"], dt)
        s["residual"] = torch.randn((M, K), generator=gen, device=dev).to(dt) if case["residual"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _plain_weights(packed, K, N, G, dt):
    """Packed buffers [n, bytes] -> W [n, K, N] in 32 bits."""
    Np, G, unit, words = _sizes(K, N, G)
    n, nb = packed.shape[0], K * Np // 2
    # block [column block, row block, lane quarter h, column c, word i]: rows 32 i + 8 h + e
    w = packed[:, :nb].contiguous().view(torch.int32).view(n, Np // 16, K // 128, 4, 16, 4)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=packed.device, dtype=torch.int32)
    q = (w[..., None] >> shift) & 15
    q = q.permute(0, 2, 5, 3, 6, 1, 4).reshape(n, K, Np)[:, :, :N].float()
    meta = packed[:, nb:].contiguous().view(torch.int32).view(n, Np, words)[:, :N, :K // unit]
    z = ((meta >> 16) & 15).transpose(1, 2).float()
    sc = (meta & 0xFFFF).to(torch.int16).view(dt).transpose(1, 2).float()
    q = q.view(n, K // unit, unit, N)
    return ((q - z[:, :, None, :]) * sc[:, :, None, :]).view(n, K, N)


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_route(s):
    case = s["case"]
    l = s["x"].double() @ s["router"].double().t()
    if case["score"] == "softmax":
        e = torch.exp(l - l.max(dim=1, keepdim=True).values)
        score = e / e.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    by = l if s["bias"] is None else score + s["bias"].double()
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :case["T"]]
    w = score.gather(1, ids)
    if case["normalize"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids.to(torch.int32), (w * case["scale"]).float()


def _plain_moe(s, ids, weights):
    case = s["case"]
    K, F, G, E, dt = case["K"], case["F"], case["G"], case["E"], _DT[case["dtype"]]
    x = s["x"].float()
    M, T = ids.shape
    ok = (ids >= 0) & (ids < E)
    at, w = ids.long().clamp(0, E - 1), weights * ok
    if M * T <= E:                 # few: the chosen experts alone, one for each entry
        pick = at.reshape(-1)
        rows = x[:, None, None, :].expand(M, T, 1, K).reshape(M * T, 1, K)
        g = torch.matmul(rows, _plain_weights(s["gate_up"][pick], K, 2 * F, G, dt))
        h = _act(case["act"], g[..., :F]) * g[..., F:]
        o = torch.matmul(h, _plain_weights(s["down"][pick], F, K, G, dt)).view(M, T, K)
        y = (o * w[:, :, None]).sum(dim=1)
    else:                          # every expert for every row, weighed by 0 where it was not chosen
        share = torch.zeros((M, E), device=x.device).scatter_add_(1, at, w)
        g = torch.matmul(x, _plain_weights(s["gate_up"], K, 2 * F, G, dt))
        h = _act(case["act"], g[..., :F]) * g[..., F:]
        y = torch.matmul(h * share.t()[:, :, None], _plain_weights(s["down"], F, K, G, dt)).sum(dim=0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt)


def _column(v, M, z):
    """A setting as [M, 1] in 64 bits."""
    return v.double()[:, None] if isinstance(v, torch.Tensor) else torch.full((M, 1), float(v), dtype=torch.float64, device=z.device)


def _plain_sample(s):
    z = s["logits"].double()
    M, V = z.shape
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    t, k, p, min_p = (_column(s[n], M, z) for n in ("t", "k", "p", "min_p"))
    p, min_p = p.float().double(), min_p.float().double()            # settings are 32-bit numbers
    t = t.float().double()
    sz, order = torch.sort(z, dim=1, descending=True, stable=True)   # ties: the lowest index first
    top = sz[:, :1]
    w = torch.where(sz == top, torch.ones_like(sz), torch.exp((sz - top) / torch.where(t > 0, t, torch.ones_like(t))))
    rank = torch.arange(V, device=z.device)[None, :]
    k = torch.where((k <= 0) | (k > V), torch.full_like(k, V), k)
    w = w * (rank < torch.where(t > 0, k, torch.ones_like(k)))       # temperature 0: the largest alone
    before = torch.cumsum(w, dim=1) - w
    cut = (p < 1) & (before >= p * w.sum(dim=1, keepdim=True)) & (rank > 0)
    w = torch.where(cut | (w < min_p.clamp(max=1.0)), torch.zeros_like(w), w)
    w = torch.zeros_like(w).scatter_(1, order, w)                    # back in index order
    total = w.sum(dim=1, keepdim=True)
    u = s["u"].double()[:, None]
    ids = (torch.cumsum(w, dim=1) <= u * total).sum(dim=1, keepdim=True).clamp(max=V - 1)
    logprob = torch.log(w.gather(1, ids) / total)
    none = top == -math.inf
    ids = torch.where(none, torch.full_like(ids, -1), ids)
    logprob = torch.where(none, torch.full_like(logprob, -math.inf), logprob)
    return ids[:, 0].to(torch.int32), logprob[:, 0].float()


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "sample":
            return _plain_sample(state)
        if op == "moe":
            return _plain_moe(state, state["ids"], state["weights"])
        ids, weights = _plain_route(state)
        return (ids, weights) if op == "route" else (_plain_moe(state, ids, weights), ids, weights)
    import w4a16_int4_weight_amd as w
    if op == "sample":
        return w.w4a16_sample(state["logits"], state["u"], temperature=state["t"], top_k=state["k"], top_p=state["p"], min_p=state["min_p"])
    if op == "moe":
        return w.w4a16_moe(state["x"], state["ids"], state["weights"], state["gate_up"], state["down"], case["F"], case["G"],
                           act=case["act"], residual=state["residual"])
    if op == "route":
        return w.w4a16_route(state["x"], state["router"], case["T"], bias=state["bias"], score=case["score"],
                             normalize=case["normalize"], scale=case["scale"])
    return w.w4a16_moe_layer(state["x"], state["router"], state["gate_up"], state["down"], case["F"], case["T"], case["G"],
                             act=case["act"], bias=state["bias"], score=case["score"], normalize=case["normalize"],
                             scale=case["scale"], residual=state["residual"])


def work(case):
    M = case["M"]
    if case["op"] == "sample":
        # each logit is read once; its difference from the largest, exponential and sum
        return {"bytes": M * case["V"] * (4 if case["dtype"] == "fp32" else 2) + 12 * M, "flops": 4.0 * M * case["V"]}
    K, E, T = case["K"], case["E"], case["T"]
    nbytes = flops = 0.0
    if case["op"] != "moe":
        nbytes += 2 * E * K + 8 * M * T
        flops += 2.0 * M * K * E
    if case["op"] == "route":
        return {"bytes": nbytes + 2 * M * K, "flops": flops}
    F = case["F"]
    # experts that some row is expected to choose: codes, one 16-bit scale and one 4-bit zero point per column and group
    used = E * (1.0 - (1.0 - T / E) ** M)
    Gu, Gd = (K if case["G"] == -1 else case["G"]), (F if case["G"] == -1 else case["G"])
    expert = 1.5 * K * F + 2.5 * (K // Gu * 2 * F + F // Gd * K)
    rows = 2 * M * K * (3 if case["residual"] else 2) + (8 * M * T if case["op"] == "moe" else 0)
    return {"bytes": nbytes + used * expert + rows, "flops": flops + 6.0 * M * T * K * F}


# ------------------------------------------------------------------ 64 bits, from the definition

def _exact_weight(packed, K, N, G, dt):
    """W^T [N, K] of one packed buffer by address, one lookup each, in 64 bits."""
    Np, G, unit, words = _sizes(K, N, G)
    k = torch.arange(K, device=packed.device)
    row, sub = k // 128, k % 128
    within = ((sub % 32) // 8) * 256 + (sub // 32) * 4          # byte of the word in its 1 KiB block, column 0
    pos = k % 8
    nibble = torch.where(pos % 2 == 0, pos // 2, 4 + pos // 2)
    n = torch.arange(N, device=packed.device)[:, None]
    byte = ((n // 16) * (K // 128) + row) * 1024 + within + (n % 16) * 16 + nibble // 2
    q = (packed[byte] >> (4 * (nibble % 2)).to(torch.uint8)) & 15
    m = K * Np // 2 + 4 * (n * words + k // unit)
    z = packed[m + 2] & 15
    bits = packed[m].to(torch.int32) | (packed[m + 1].to(torch.int32) << 8)
    return (q.double() - z.double()) * bits.to(torch.int16).view(dt).double()


def _exact_route(s):
    case = s["case"]
    l = torch.stack([(s["router"].double() * row).sum(dim=1) for row in s["x"].double()])
    score = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)
    by = (l if s["bias"] is None else score + s["bias"].double()).clone()
    ids = []
    for _ in range(case["T"]):
        best = by.max(dim=1, keepdim=True).values
        ids.append((by == best).to(torch.int8).argmax(dim=1, keepdim=True))
        by.scatter_(1, ids[-1], -math.inf)
    ids = torch.cat(ids, dim=1)
    w = score.gather(1, ids)
    if case["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w * case["scale"]


def _exact_moe(s, ids, weights):
    case = s["case"]
    K, F, dt = case["K"], case["F"], _DT[case["dtype"]]
    x = s["x"].double()
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    for e in range(case["E"]):
        hit = ids == e
        rows = hit.any(dim=1).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        up = x[rows] @ _exact_weight(s["gate_up"][e], K, 2 * F, case["G"], dt).t()
        g, u = up[:, :F], up[:, F:]
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            a = 0.5 * g * torch.erfc(-g * math.sqrt(0.5))
        else:
            a = g * torch.sigmoid(2 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
        o = (a * u) @ _exact_weight(s["down"][e], F, K, case["G"], dt).t()
        y[rows] += (weights.double() * hit).sum(dim=1)[rows, None] * o
    return y


def _exact_sample(s):
    z = s["logits"].double()
    M, V = z.shape
    ids = torch.full((M,), -1, dtype=torch.int32, device=z.device)
    logprob = torch.full((M,), -math.inf, dtype=torch.float64, device=z.device)
    row = lambda v, m: float(v[m]) if isinstance(v, torch.Tensor) else float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    for m in range(M):
        t, k, p, min_p = (row(s[n], m) for n in ("t", "k", "p", "min_p"))
        live = (z[m] > -math.inf).nonzero()[:, 0]              # in index order
        if live.numel() == 0:
            continue
        if t <= 0:
            k, t = 1, 1.0
        l = z[m][live]
        w = torch.exp((l - l.max()) / t)
        order = torch.sort(-l, stable=True).indices            # falling, ties lowest index first
        if 0 < k < live.numel():
            order = order[:int(k)]
        sums = torch.cumsum(w[order], dim=0)
        if p < 1:
            order = order[:int((sums < p * sums[-1]).sum()) + 1]
        order = order[w[order] >= min(min_p, 1.0)]
        kept = order.sort().values
        sums = torch.cumsum(w[kept], dim=0)
        j = int((sums <= float(s["u"][m]) * sums[-1]).sum())
        ids[m] = live[kept[j]].to(torch.int32)
        logprob[m] = torch.log(w[kept[j]] / sums[-1])
    return ids, logprob


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "moe":
        return _exact_moe(s, s["ids"], s["weights"])
    ids, weights = _exact_route(s)
    return (ids, weights) if case["op"] == "route" else (_exact_moe(s, ids, weights), ids, weights)
