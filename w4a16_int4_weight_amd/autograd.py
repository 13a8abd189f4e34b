"""The operators on frozen packed int4 weights as differentiable torch operations.

  linear(x, packed, N, group_size, bias)                    -> y = x W (+ bias)
  gated(x, packed, F, group_size, act)                      -> h = a(x Wg) * (x Wu)
  cross_entropy(x, labels, packed, V, group_size, weights)  -> weights[m] * loss[m]
  distill(x, top_ids, top_logits, packed, V, group_size, temperature, weights)

Gradients go to x alone: the weights, a bias, the rows' weights and a teacher's logits are
constants, and ValueError is raised for one that requires a gradient (detach it). x is
fp16 or bf16, [..., K]; a dimension of any size is met as rows. Each call runs on the
current stream, like the functions it is made of.

The losses form x's gradient in the forward pass, where the head is read for the loss
anyway (not under no_grad, or for an x that requires none), scaled by `weights` (float32 per row; None: 1). Give the rows' weights there
(1 / count for a mean) and sum what comes back: the backward pass then multiplies by one,
which is exact. A power of two on the loss (a gradient scaler's) is exact too; another
factor on a row is one more rounding. fp16 keeps the gradient at its weight's mantissa and
takes the weight's power of two into the backward pass, with the loss's own factor: what
1 / count makes too small for fp16 is whole again under a loss scale.
"""

import torch

from . import _beside, w4a16_cross_entropy, w4a16_distill, w4a16_gated, w4a16_gated_grad, w4a16_gemm, w4a16_gemm_grad

__all__ = ["linear", "gated", "cross_entropy", "distill"]


def _flat(x):
    return x.reshape(-1, x.shape[-1]).contiguous()


def _constant(t, name):
    if t is not None and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} is a constant here and gets no gradient: detach it")
    return t


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, packed, N, group_size, bias):
        ctx.save_for_backward(packed)
        ctx.shape, ctx.group_size = x.shape, group_size
        return w4a16_gemm(_flat(x), packed, N, group_size, bias=bias).view(*x.shape[:-1], N)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        packed, = ctx.saved_tensors
        dx = w4a16_gemm_grad(_flat(dy), packed, ctx.shape[-1], ctx.group_size)
        return dx.view(ctx.shape), None, None, None, None


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, packed, F, group_size, act):
        flat = _flat(x)
        ctx.save_for_backward(flat, packed)
        ctx.shape, ctx.args = x.shape, (F, group_size, act)
        return w4a16_gated(flat, packed, F, group_size, act=act).view(*x.shape[:-1], F)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        flat, packed = ctx.saved_tensors
        F, group_size, act = ctx.args
        dx = w4a16_gated_grad(flat, _flat(dh), packed, F, group_size, act=act)
        return dx.view(ctx.shape), None, None, None, None


class _Loss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weights, call, grad):
        flat = _flat(x)
        if weights is not None:
            weights = weights.reshape(-1).contiguous()
        dloss, power = weights, None
        if grad and weights is not None and x.dtype == torch.float16:
            dloss, power = torch.frexp(weights)
        out = call(flat, grad, dloss if grad else None)
        ctx.shape = x.shape
        if grad:
            ctx.save_for_backward(out[2], power)
        loss = out[0] if weights is None else out[0] * weights
        return loss.view(x.shape[:-1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        dx, power = ctx.saved_tensors
        g = g.reshape(-1)
        if power is not None:
            g = torch.ldexp(g, power)
        return (dx.float() * g[:, None]).to(dx.dtype).view(ctx.shape), None, None, None


def _loss(x, weights, call):
    # (asked here: inside a Function an x that requires a gradient says so under no_grad too)
    return _Loss.apply(x, _constant(weights, "weights"), call, x.requires_grad and torch.is_grad_enabled())


def linear(x, packed, N, group_size=128, bias=None):
    """w4a16_gemm, with w4a16_gemm_grad as its backward pass."""
    _beside(x, packed=packed, bias=bias)
    return _Linear.apply(x, packed, N, group_size, _constant(bias, "bias"))


def gated(x, packed, F, group_size=128, act="silu"):
    """w4a16_gated, with w4a16_gated_grad as its backward pass (x is kept, not g and u)."""
    return _Gated.apply(x, packed, F, group_size, act)


def cross_entropy(x, labels, packed, V, group_size=128, weights=None):
    """w4a16_cross_entropy: weights[m] * loss[m], float32, shaped like labels. labels int32;
    a label outside [0, V) has loss and gradient 0."""
    def call(flat, grad, dloss):
        return w4a16_cross_entropy(flat, labels.reshape(-1).contiguous(), packed, V, group_size, dloss=dloss, grad=grad)
    return _loss(x, weights, call)


def distill(x, top_ids, top_logits, packed, V, group_size=128, temperature=1.0, weights=None):
    """w4a16_distill: weights[m] * loss[m], float32. top_ids, top_logits [..., T]."""
    _constant(top_logits, "top_logits")

    def call(flat, grad, dloss):
        return w4a16_distill(flat, _flat(top_ids), _flat(top_logits), packed, V, group_size, temperature=temperature,
                             dloss=dloss, grad=grad)
    return _loss(x, weights, call)
