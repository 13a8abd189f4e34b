"""Plain 64-bit forms of the router, the experts' layer and the draw of a token, written from
their definitions."""

import numpy as np
import torch

import train_util as tu
from gpu_util import DEV, TORCH_DTYPE

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}      # of a rounding, relative to the value


class Experts:
    """E seeded experts: packed buffers [E, bytes] on the device and their exact values."""

    def __init__(self, w, seed, E, K, F, dtype, group_size, pad=0):
        up = [tu.Weight(w, seed + 2 * e, K, 2 * F, dtype, group_size) for e in range(E)]
        down = [tu.Weight(w, seed + 2 * e + 1, F, K, dtype, group_size) for e in range(E)]
        self.E, self.K, self.F, self.G, self.dtype = E, K, F, group_size, dtype
        self.up, self.down = [t.dev64 for t in up], [t.dev64 for t in down]

        def stack(ts):
            n = ts[0].packed.numel()
            out = torch.full((E, n + pad), 255, dtype=torch.uint8, device=DEV)    # a stride beyond the weight
            for e, t in enumerate(ts):
                out[e, :n] = t.packed
            return out
        self.gate_up, self.down_packed = stack(up), stack(down)


def moe(ex, x, ids, weights, act="silu", residual=None):
    """x, weights float64 on the device; ids int [M, T] -> y float64 [M, K]"""
    y = torch.zeros_like(x) if residual is None else residual.clone()
    for e in range(ex.E):
        hit = ids == e
        rows = hit.any(dim=1).nonzero()[:, 0]
        if rows.numel():
            o = tu.gated(ex.up[e], ex.F, x[rows], act) @ ex.down[e]
            y[rows] += (torch.where(hit, weights, torch.zeros_like(weights)).sum(dim=1))[rows, None] * o
    return y


def check_moe(got, ref, dtype):
    """One rounding to dtype: half a step of the value at each element (its norm: that over
    sqrt(3) for evenly spread values); what the fp32 sums and h's 16 bits lose before it is
    below 2e-5 in the norm, five times that at an element."""
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all()
    half = HALF_STEP[dtype]
    rms = float(ref.norm()) / max(1, ref.numel()) ** 0.5
    over = (got - ref).abs() - half * ref.abs() - 1e-4 * rms
    assert float(over.max()) <= 0, f"element off by {float(over.max())} beyond its bound, rms {rms}"
    if ref.numel() >= 1024:
        assert tu.norm_err(got, ref) <= half / 3 ** 0.5 * 1.05 + 2e-5


def route(x, router, T, bias=None, score="softmax", normalize=True, scale=1.0):
    """float64 x [M, K], router [E, K] -> ids [M, T], weights float64 [M, T]"""
    l = (x[:, None, :] * router[None, :, :]).sum(-1)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    by = l if bias is None else s + bias.double()
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :T]
    w = s.gather(1, ids)
    if normalize:
        w = w / w.sum(1, keepdim=True)
    return ids, w * scale


def sample(logits, u, t=1.0, k=0, p=1.0, min_p=0.0):
    """Row by row in NumPy float64. Settings: numbers or float32/int32 arrays [M]."""
    z = logits.detach().double().cpu().numpy()
    u = u.detach().double().cpu().numpy()
    M, V = z.shape
    ids, logprob = np.full(M, -1), np.full(M, -np.inf)

    def of(v, m):
        if isinstance(v, torch.Tensor):
            return float(v[m])
        return float(np.float32(v))
    for m in range(M):
        zr = np.where(np.isnan(z[m]), -np.inf, z[m])
        top = zr.max()
        if top == -np.inf:
            continue
        tt, kk, pp, mp = of(t, m), int(of(k, m)), of(p, m), of(min_p, m)
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.where(zr == top, 1.0, np.where(zr == -np.inf, 0.0, np.exp((zr - top) / (tt if tt > 0 else 1.0))))
        order = np.lexsort((np.arange(V), -zr))              # falling, ties lowest index first
        if not tt > 0:
            kk, pp, mp = 1, 1.0, 0.0
        if 1 <= kk < V:
            order = order[:kk]
        if pp < 1:
            before = np.cumsum(w[order]) - w[order]
            n = int((before < max(pp, 0.0) * w[order].sum()).sum())
            order = order[:max(n, 1)]
        if mp > 0:
            order = order[w[order] >= min(mp, 1.0)]
        kept = np.sort(order)
        run = np.cumsum(w[kept])
        uu = u[m] if u[m] > 0 else 0.0
        j = int(np.searchsorted(run, uu * run[-1], side="right"))
        if j >= len(kept):
            j = int(np.nonzero(w[kept] > 0)[0][-1])
        ids[m] = kept[j]
        logprob[m] = np.log(w[kept[j]] / run[-1])
    return ids, logprob


def to64(t):
    return t.double()


def dt(name):
    return torch.float32 if name == "fp32" else TORCH_DTYPE[name]
