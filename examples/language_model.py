"""Training a small language model with shared embedding and head weights, every kernel this library's own:

    tokens -> embedding -> layer norm -> linear + GELU -> linear + residual -> layer norm
      -> cross entropy over the vocabulary, without its logits -> backward -> clipped AdamW step

The table serves as the head's weight too: the head's gradient is made first
and the embedding's is added to it.  Matrices are bf16 copies of fp32 master
weights; their moments are held in 8 bits, those of the norms and biases in 32.
The texts are sequences of a random order: a token is mostly followed by the
same few others.

    python examples/language_model.py [--steps 200] [--width 512] [--vocab 8000]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from tensor_grad_clip_gb300 import SomaOpt, TensorList, ops, zeros_8bit  # noqa: E402


class Model:
    def __init__(self, width: int, vocab: int, device, seed: int):
        gen = torch.Generator(device=device).manual_seed(seed)

        def matrix(n, k, std):
            return torch.randn(n, k, device=device, generator=gen) * std
        one, zero = torch.ones(width, device=device), torch.zeros(width, device=device)
        # fp32 master weights; matrices and their biases have a bf16 copy that the model runs on
        self.masters = {
            "table": matrix(vocab, width, 0.05), "in.weight": one, "in.bias": zero,
            "up.weight": matrix(4 * width, width, width ** -0.5), "up.bias": torch.zeros(4 * width, device=device),
            "down.weight": matrix(width, 4 * width, 0.5 * (4 * width) ** -0.5), "down.bias": zero.clone(),
            "out.weight": one.clone(), "out.bias": zero.clone(),
        }
        self.model = {k: v if k.startswith(("in.", "out.")) else v.bfloat16() for k, v in self.masters.items()}
        self.scale = math.sqrt(width)

    def loss_and_gradients(self, texts, weight):
        """The loss of each position (the next token's cross entropy, times `weight`) and all weights' gradients."""
        w, g = self.model, {}
        tokens, targets = texts[:, :-1], texts[:, 1:]
        x = ops.embedding_forward(tokens, w["table"], scale=self.scale)
        h, mean, rstd = ops.layer_norm_forward(x, w["in.weight"], w["in.bias"])
        u, z = ops.linear_forward(h, w["up.weight"], w["up.bias"], activation="gelu", save_preactivation=True)
        y = ops.linear_forward(u, w["down.weight"], w["down.bias"], residual=x)
        o, mean2, rstd2 = ops.layer_norm_forward(y, w["out.weight"], w["out.bias"])
        loss, do, g["table"] = ops.linear_cross_entropy_loss_grad(o, w["table"], targets, row_weight=weight)
        dy, g["out.weight"], g["out.bias"] = ops.layer_norm_backward(do, y, w["out.weight"], mean2, rstd2)
        du, g["down.weight"], g["down.bias"] = ops.linear_backward(dy, u, w["down.weight"])
        dh, g["up.weight"], g["up.bias"] = ops.linear_backward(du, h, w["up.weight"], z, activation="gelu")
        dx, g["in.weight"], g["in.bias"] = ops.layer_norm_backward(dh, x, w["in.weight"], mean, rstd)
        ops.embedding_backward(dx.add_(dy), tokens, len(w["table"]), scale=self.scale, out=g["table"])
        return loss, g


class Trainer:
    def __init__(self, model: Model, lr: float, weight_decay: float = 0.01, max_norm: float = 1.0):
        self.model, self.max_norm, self.names = model, max_norm, list(model.masters)
        self.opt = SomaOpt(device=model.masters["table"].device.index)
        decayed, plain = self.opt.add_group(lr=lr, weight_decay=weight_decay), self.opt.add_group(lr=lr)
        self.groups, self.moments = [], []  # (m, v) as (values, scales) each
        for k in self.names:
            p = model.masters[k]
            matrix = p.dim() == 2
            self.groups.append(decayed if matrix else plain)
            self.moments.append([zeros_8bit(p) if matrix else (torch.zeros_like(p), None) for _ in range(2)])

    def step(self, texts):
        """One step on a batch of texts; returns the mean loss per position (a device tensor) and the gradients."""
        weight = torch.full((texts.shape[0], texts.shape[1] - 1), 1.0 / (texts.shape[0] * (texts.shape[1] - 1)),
                            device=texts.device)
        loss, grads = self.model.loss_and_gradients(texts, weight)
        masters, model, names = self.model.masters, self.model.model, self.names
        m, v = zip(*self.moments)
        tensors = TensorList([masters[k] for k in names], [grads[k] for k in names], [x[0] for x in m], [x[0] for x in v],
                             self.groups, params_lowp=[None if model[k] is masters[k] else model[k] for k in names],
                             exp_avg_scales=[x[1] for x in m], exp_avg_sq_scales=[x[1] for x in v])
        self.opt.step(tensors, grad_divisor=1.0, max_norm=self.max_norm)
        return loss.sum(), grads


def texts_of(order, batch: int, length: int, gen):
    """Texts in which one of a token's `order.shape[1]` followers comes next."""
    vocab, followers = order.shape
    text = torch.empty(batch, length, dtype=torch.int64, device=order.device)
    text[:, 0] = torch.randint(0, vocab, (batch,), device=order.device, generator=gen)
    for i in range(1, length):
        pick = torch.randint(0, followers, (batch,), device=order.device, generator=gen)
        text[:, i] = order[text[:, i - 1], pick]
    return text


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=64, help="texts per step")
    ap.add_argument("--length", type=int, default=65, help="tokens of a text")
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=8000)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args(argv)
    device = torch.device("cuda", 0)
    gen = torch.Generator(device=device).manual_seed(3)
    order = torch.randint(0, a.vocab, (a.vocab, 4), device=device, generator=gen)
    trainer = Trainer(Model(a.width, a.vocab, device, seed=1), a.lr)
    losses = []
    for step in range(a.steps):
        loss, _ = trainer.step(texts_of(order, a.batch, a.length, gen))
        losses.append(loss)
        if step % 20 == 0 or step == a.steps - 1:
            norm, coef, _ = trainer.opt.get_norm()
            print(f"step {step:4d}  loss {loss.item():.4f}  gradient norm {norm:.4f}  clip coefficient {coef:.4f}")
    return [v.item() for v in losses]


if __name__ == "__main__":
    main()
