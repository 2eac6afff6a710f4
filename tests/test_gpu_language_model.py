"""The language model's operators together, as examples/language_model.py uses them: one step's gradients against fp64, and
that it runs."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("width,vocab,batch,length", [(64, 300, 5, 9), (96, 1001, 20, 33)])
def test_gradients_of_one_step(example, width, vocab, batch, length):
    dev = torch.device("cuda", 0)
    torch.manual_seed(1)
    model = example.Model(width, vocab, dev, seed=2)
    texts = torch.randint(0, vocab, (batch, length), device=dev)
    texts[0, 4:] = -1   # a short text: neither looked up nor predicted
    weight = torch.rand(batch, length - 1, device=dev)
    loss, grads = model.loss_and_gradients(texts, weight)
    w = {k: v.double().requires_grad_() for k, v in model.model.items()}
    tokens, targets = texts[:, :-1], texts[:, 1:]

    def norm(x, name):
        return torch.nn.functional.layer_norm(x, (width,), w[name + ".weight"], w[name + ".bias"])
    x = torch.where((tokens >= 0)[..., None], w["table"][tokens.clamp(min=0)] * math.sqrt(width), 0.0)
    h = norm(x, "in")
    y = torch.nn.functional.gelu(h @ w["up.weight"].t() + w["up.bias"]) @ w["down.weight"].t() + w["down.bias"] + x
    logits = norm(y, "out") @ w["table"].t()
    each = torch.nn.functional.cross_entropy(logits.transpose(1, 2), targets, ignore_index=-1, reduction="none")
    want = (each * weight).sum()
    want.backward()
    # a handful of roundings to bf16 (2^-8 each) lie between any weight and the loss
    assert abs(loss.sum().item() - want.item()) <= 2 ** -6 * abs(want.item())
    assert not loss[0, 3:].any()
    for k, v in w.items():
        off = (grads[k].double() - v.grad).norm() / v.grad.norm()
        assert off <= 8 * 2 ** -8, (k, float(off))


def test_a_step_changes_every_weight(example):
    dev = torch.device("cuda", 0)
    trainer = example.Trainer(example.Model(64, 200, dev, seed=2), lr=1e-3)
    masters = {k: v.clone() for k, v in trainer.model.masters.items()}
    trainer.step(torch.randint(0, 200, (8, 17), device=dev))
    for k, v in trainer.model.masters.items():
        assert not torch.equal(v, masters[k]), k
        if v.dim() == 2:
            assert torch.equal(trainer.model.model[k], v.bfloat16()), k


def test_it_runs(example, capsys):
    losses = example.main(["--steps", "25", "--batch", "8", "--length", "17", "--width", "64", "--vocab", "500"])
    assert len(losses) == 25 and all(math.isfinite(v) and v > 0 for v in losses)
    assert "clip coefficient" in capsys.readouterr().out
