"""Training a small head by distillation, every kernel this library's own:

    x -> layer norm -> linear + GELU -> linear + residual -> linear to the vocabulary
      -> distillation loss from a teacher's top logits -> backward -> clipped AdamW step

The model's matrices are bf16 copies of fp32 master weights; the optimizer
step clips all gradients by their global norm, updates the masters and
rewrites the copies.  The teacher is a fixed random head of the same shape;
it answers each position with its `top` largest logits.

    python examples/distill_head.py [--steps 200] [--width 1024] [--vocab 32000]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from tensor_grad_clip_gb300 import SomaOpt, TensorList, ops  # noqa: E402


class Head:
    """Weights of one residual block and the projection to the vocabulary."""

    def __init__(self, width: int, vocab: int, device, seed: int):
        gen = torch.Generator(device=device).manual_seed(seed)

        def matrix(n, k):
            return torch.randn(n, k, device=device, generator=gen) / math.sqrt(k)
        # fp32 master weights; matrices and their biases have a bf16 copy that the model runs on
        self.masters = {
            "norm.weight": torch.ones(width, device=device), "norm.bias": torch.zeros(width, device=device),
            "up.weight": matrix(4 * width, width), "up.bias": torch.zeros(4 * width, device=device),
            "down.weight": matrix(width, 4 * width), "down.bias": torch.zeros(width, device=device),
            "out.weight": matrix(vocab, width),
        }
        self.model = {k: v if k.startswith("norm") else v.bfloat16() for k, v in self.masters.items()}

    def forward(self, x):
        """Logits, and what the backward pass needs."""
        w = self.model
        h, mean, rstd = ops.layer_norm_forward(x, w["norm.weight"], w["norm.bias"])
        u, z = ops.linear_forward(h, w["up.weight"], w["up.bias"], activation="gelu", save_preactivation=True)
        y = ops.linear_forward(u, w["down.weight"], w["down.bias"], residual=x)
        return ops.linear_forward(y, w["out.weight"]), (x, mean, rstd, h, u, z, y)

    def backward(self, dlogits, saved):
        """Gradients of all weights (matrices in bf16, the norm's in fp32)."""
        w, (x, mean, rstd, h, u, z, y) = self.model, saved
        g = {}
        dy, g["out.weight"], _ = ops.linear_backward(dlogits, y, w["out.weight"], bias_grad=False)
        du, g["down.weight"], g["down.bias"] = ops.linear_backward(dy, u, w["down.weight"])
        dh, g["up.weight"], g["up.bias"] = ops.linear_backward(du, h, w["up.weight"], z, activation="gelu")
        _, g["norm.weight"], g["norm.bias"] = ops.layer_norm_backward(dh, x, w["norm.weight"], mean, rstd,
                                                                      input_grad=False)
        return g


class Trainer:
    def __init__(self, head: Head, lr: float, weight_decay: float = 0.01, max_norm: float = 1.0):
        self.head, self.max_norm, self.names = head, max_norm, list(head.masters)
        self.opt = SomaOpt(device=head.masters["norm.weight"].device.index)
        decayed, plain = self.opt.add_group(lr=lr, weight_decay=weight_decay), self.opt.add_group(lr=lr)
        self.groups = [decayed if head.masters[k].dim() == 2 else plain for k in self.names]
        self.moments = [{k: torch.zeros_like(v) for k, v in head.masters.items()} for _ in range(2)]

    def step(self, x, teacher_logits, teacher_index, temperature: float):
        """One step on a batch; returns the mean loss per position (a device tensor)."""
        logits, saved = self.head.forward(x)
        weight = torch.full(logits.shape[:-1], 1.0 / logits[..., 0].numel(), device=x.device)
        # the gradient takes the logits' place
        loss, dlogits = ops.distill_loss_grad(logits, teacher_logits, teacher_index, temperature=temperature,
                                              row_weight=weight, out=logits)
        grads = self.head.backward(dlogits, saved)
        masters, model, names = self.head.masters, self.head.model, self.names
        # The handle keeps the tables of the last few lists of buffers that it
        # stepped; the allocator usually hands the gradients the same memory again.
        tensors = TensorList([masters[k] for k in names], [grads[k] for k in names],
                             [self.moments[0][k] for k in names], [self.moments[1][k] for k in names], self.groups,
                             params_lowp=[None if model[k] is masters[k] else model[k] for k in names])
        self.opt.step(tensors, grad_divisor=1.0, max_norm=self.max_norm)
        return loss.sum(), grads


def teacher_answers(teacher: Head, x, top: int):
    logits, _ = teacher.forward(x)
    values, index = logits.float().topk(top, dim=-1)
    return values, index.int()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=2048, help="positions per step")
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--top", type=int, default=64)
    ap.add_argument("--temperature", type=float, default=2.0)
    ap.add_argument("--lr", type=float, default=4e-3)
    a = ap.parse_args(argv)
    device = torch.device("cuda", 0)
    teacher, trainer = Head(a.width, a.vocab, device, seed=1), Trainer(Head(a.width, a.vocab, device, seed=2), a.lr)
    gen = torch.Generator(device=device).manual_seed(3)
    losses = []
    for step in range(a.steps):
        x = torch.randn(a.batch, a.width, device=device, generator=gen).bfloat16()
        loss, _ = trainer.step(x, *teacher_answers(teacher, x, a.top), temperature=a.temperature)
        losses.append(loss)
        if step % 20 == 0 or step == a.steps - 1:
            norm, coef, _ = trainer.opt.get_norm()
            print(f"step {step:4d}  loss {loss.item():.4f}  gradient norm {norm:.4f}  clip coefficient {coef:.4f}")
    return [v.item() for v in losses]


if __name__ == "__main__":
    main()
