"""Plain 64-bit forms of the training operators, written from their definitions with
NumPy (or, at sizes NumPy is slow for, float64 torch on the GPU), on weights decoded from
the checkpoint tensors by the oracle."""

import numpy as np
import torch

import synth
from oracle import awq, gemm as ogemm, numerics
from gpu_util import DEV, bits_to_device, weights_to_device

ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}     # half a step, relative to the value


class Weight:
    """A seeded packed weight on the device, and its exact values in float64 [K, N]."""

    def __init__(self, w, seed, K, N, dtype, group_size):
        ws = synth.make_custom(seed, 1, K, N, dtype, group_size)
        self.K, self.N, self.dtype, self.G = K, N, dtype, group_size
        qw, qz, sc = weights_to_device(ws)
        self.packed = w.w4a16_repack(qw, qz, sc, group_size)
        self.W = ogemm.dequant(awq.unpack_awq(ws.qweight), awq.unpack_awq(ws.qzeros),
                                numerics.half_bits_to_f64(ws.scale_bits, dtype), group_size)
        self.dev64 = torch.from_numpy(np.ascontiguousarray(self.W)).to(DEV)


def normal(seed, shape, dtype, scale=1.0):
    """-> (device tensor of dtype, the same values in float64 on the device)"""
    rng = np.random.default_rng(seed)
    bits = synth.f32_to_half_bits((rng.standard_normal(shape) * scale).astype(np.float32), dtype)
    t = bits_to_device(bits, dtype)
    return t, t.double()


def act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return 0.5 * g * torch.erfc(-g / np.sqrt(2.0))
    return 0.5 * g * (1 + torch.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def gated(W, F, x, name):
    g, u = x @ W[:, :F], x @ W[:, F:]
    return act(name, g) * u


def gated_grad(W, F, x, dh, name):
    x = x.clone().requires_grad_(True)
    return torch.autograd.grad(gated(W, F, x, name), x, dh)[0]


def targets(ids, weights, V):
    """dense [M, V] target weights; ids outside [0, V) dropped"""
    M, T = ids.shape
    d = torch.zeros((M, V), dtype=torch.float64, device=ids.device)
    ok = (ids >= 0) & (ids < V)
    return d.scatter_add_(1, ids.clamp(0, V - 1).long(), weights * ok)


def teacher(ids, t, V, tau):
    ok = (ids >= 0) & (ids < V)
    v = torch.where(ok, t.double() / tau, torch.full_like(t, -np.inf, dtype=torch.float64))
    top = v.max(dim=1, keepdim=True).values
    e = torch.exp(v - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    s = e.sum(1, keepdim=True)
    return e / torch.where(s == 0, torch.ones_like(s), s)


def loss(W, x, ids, p, tau, dloss):
    """-> (loss, lse, dx, z) for entry weights p [M, T]"""
    V = W.shape[1]
    z = (x @ W) / tau
    lse = torch.logsumexp(z, dim=1)
    ok = (ids >= 0) & (ids < V)
    zt = z.gather(1, ids.clamp(0, V - 1).long())
    some = (p * ok).sum(1) > 0
    terms = torch.special.xlogy(p, p) - torch.where(p * ok > 0, p * (zt - lse[:, None]), torch.zeros_like(p))
    value = torch.where(some, tau * tau * (terms * ok).sum(1), torch.zeros_like(lse))
    d = torch.softmax(z, 1) - targets(ids, p, V)
    d = torch.where(some[:, None], d, torch.zeros_like(d))
    dx = torch.where(some, tau * dloss, torch.zeros_like(dloss))[:, None] * (d @ W.t())
    return value, lse, dx, z


def norm_err(got, ref):
    """||got - ref|| / ||ref|| over the whole tensor"""
    got, ref = got.double(), ref.double()
    n = ref.norm()
    return float((got - ref).norm() / n) if float(n) else float((got - ref).norm())
