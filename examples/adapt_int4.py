"""Fine-tuning an adapter through frozen int4 weights: the operators of
w4a16_int4_weight_amd.autograd used together.

A two-layer model whose every large weight is packed int4 (per layer a gated
feed-forward block and its down projection, then the output head) learns, through a
low-rank adapter beside each layer, to follow a teacher: first by cross entropy on the
teacher's most likely tokens, then by distillation from its top logits. The teacher is
the same model with other (fixed) adapters. Last, the student's log-probabilities of a
few tokens are scored, row by row, as while serving.

    python examples/adapt_int4.py [--steps 30] [--dtype bf16]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_int4_weight_amd as w  # noqa: E402
from w4a16_int4_weight_amd import autograd as ops  # noqa: E402

K, F, V, G, RANK, LAYERS = 512, 1024, 4096, 128, 16, 2


def packed_weight(rows, cols, gen, dtype, device):
    """A random weight as a GPTQ checkpoint would bring it, packed."""
    def words(*shape):
        return torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen, dtype=torch.int64).to(torch.int32)
    scales = (torch.rand((rows // G, cols), generator=gen) * 0.5 + 0.75) / (6.5 * rows ** 0.5)
    return w.w4a16_repack_gptq(words(rows // 8, cols).to(device), words(rows // G, cols // 8).to(device),
                               scales.to(dtype).to(device), G)


class Model:
    def __init__(self, gen, dtype, device):
        self.up = [packed_weight(K, 2 * F, gen, dtype, device) for _ in range(LAYERS)]
        self.down = [packed_weight(F, K, gen, dtype, device) for _ in range(LAYERS)]
        self.head = packed_weight(K, V, gen, dtype, device)

    def features(self, x, adapters):
        for i in range(LAYERS):
            a, b = adapters[2 * i], adapters[2 * i + 1]
            h = ops.gated(x, self.up[i], F, G)
            x = x + ops.linear(h, self.down[i], K, G) + (x @ a.to(x.dtype)) @ b.to(x.dtype)
            x = (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)
        return 4 * x


def adapters(gen, device, scale):
    out = []
    for _ in range(LAYERS):
        out.append((torch.randn((K, RANK), generator=gen) / K ** 0.5).to(device))
        out.append((torch.randn((RANK, K), generator=gen) * scale).to(device))
    return out


def run(steps=30, dtype=torch.bfloat16, device="cuda:0", log=print):
    """-> (losses of the cross entropy phase, of the distillation phase, scores)"""
    gen = torch.Generator().manual_seed(0)
    model = Model(gen, dtype, device)
    x = torch.randn((256, K), generator=gen).to(dtype).to(device)
    with torch.no_grad():
        teacher = model.features(x, adapters(gen, device, 0.5))
        logits = w.w4a16_gemm(teacher.contiguous(), model.head, V, G).float()
        top_logits, top_ids = logits.topk(20, dim=1)
        top_ids, top_logits = top_ids.to(torch.int32), top_logits.contiguous()
        labels = top_ids[:, 0].contiguous()
        labels[::16] = -100                                     # rows without a label
    student = [t.requires_grad_(True) for t in adapters(gen, device, 0.0)]
    optimizer = torch.optim.Adam(student, lr=2e-2)
    scale = 128.0 if dtype == torch.float16 else 1.0            # keeps fp16 gradients in range
    weights = torch.full((x.shape[0],), scale / x.shape[0], device=device)

    history = {"cross entropy": [], "distillation": []}
    for phase, losses in history.items():
        for step in range(steps):
            y = model.features(x, student)
            if phase == "cross entropy":
                loss = ops.cross_entropy(y, labels, model.head, V, G, weights=weights).sum()
            else:
                loss = ops.distill(y, top_ids, top_logits, model.head, V, G, temperature=2.0, weights=weights).sum()
            optimizer.zero_grad()
            loss.backward()
            for p in student:
                p.grad /= scale
            optimizer.step()
            losses.append(float(loss.detach()) / scale)
        log(f"{phase}: {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    with torch.no_grad():
        y = model.features(x, student)
        scores = torch.stack([-w.w4a16_cross_entropy(y[m:m + 1], top_ids[m:m + 1, 0].contiguous(), model.head, V, G)[0][0]
                              for m in range(4)])
    log("log-probabilities of the teacher's tokens: " + ", ".join(f"{float(s):.3f}" for s in scores))
    return history["cross entropy"], history["distillation"], scores


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=30)
    parser.add_argument("--dtype", choices=["bf16", "fp16"], default="bf16")
    args = parser.parse_args()
    run(args.steps, torch.bfloat16 if args.dtype == "bf16" else torch.float16)
