"""The operators together, as examples/distill_head.py uses them: one step's
gradients against fp64, and a short training run whose loss falls."""
import importlib.util
import os

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("distill_head", os.path.join(ROOT, "examples", "distill_head.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_gradients_of_one_step(example):
    dev = torch.device("cuda", 0)
    head, teacher = example.Head(96, 1000, dev, seed=2), example.Head(96, 1000, dev, seed=1)
    x = torch.randn(77, 96, device=dev).bfloat16()
    t, index = example.teacher_answers(teacher, x, 20)
    trainer = example.Trainer(head, lr=1e-3)
    before = {k: v.double() for k, v in head.model.items()}
    masters = {k: v.clone() for k, v in head.masters.items()}
    loss, grads = trainer.step(x, t, index, temperature=2.0)
    w = {k: v.clone().requires_grad_() for k, v in before.items()}
    xd = x.double()
    mean = xd.mean(1, keepdim=True)
    h = (xd - mean) / torch.sqrt(((xd - mean) ** 2).mean(1, keepdim=True) + 1e-5) * w["norm.weight"] + w["norm.bias"]
    y = R.activate(h @ w["up.weight"].t() + w["up.bias"], "gelu") @ w["down.weight"].t() + w["down.bias"] + xd
    logits = y @ w["out.weight"].t()
    p = torch.softmax(t.double() / 2, 1)
    logq = torch.log_softmax(logits / 2, 1).gather(1, index.long())
    want = (4 * (p * (torch.log(p) - logq)).sum(1)).mean()
    want.backward()
    # a handful of roundings to bf16 (2^-8 each) lie between any weight and the loss
    assert abs(loss.item() - want.item()) <= 2 ** -6 * abs(want.item())
    for k, v in w.items():
        off = (grads[k].double() - v.grad).norm() / v.grad.norm()
        assert off <= 8 * 2 ** -8, (k, float(off))
        assert not torch.equal(head.masters[k], masters[k]), f"{k} was not updated"
        assert torch.equal(head.model[k], head.masters[k].to(head.model[k].dtype))


def test_the_loss_falls(example, capsys):
    losses = example.main(["--steps", "60", "--batch", "512", "--width", "128", "--vocab", "2000", "--top", "32"])
    assert all(v == v and v >= 0 for v in losses)
    assert sum(losses[-10:]) < 0.7 * sum(losses[:10])
    assert "clip coefficient" in capsys.readouterr().out


def test_autograd_gives_the_same_gradients(example):
    from tensor_grad_clip_gb300 import ops
    dev = torch.device("cuda", 0)
    head, teacher = example.Head(64, 700, dev, seed=2), example.Head(64, 700, dev, seed=1)
    x = torch.randn(33, 64, device=dev).bfloat16()
    t, index = example.teacher_answers(teacher, x, 9)
    logits, saved = head.forward(x)
    loss, lse = ops.distill_forward(logits, t, index, temperature=2.0)
    d = ops.distill_backward(torch.ones_like(loss), logits, lse, t, index, temperature=2.0)
    grads = head.backward(d, saved)
    w = {k: v.clone().requires_grad_() for k, v in head.model.items()}
    h = ops.layer_norm(x, w["norm.weight"], w["norm.bias"])
    u = ops.linear(h, w["up.weight"], w["up.bias"], activation="gelu")
    y = ops.linear(u, w["down.weight"], w["down.bias"], residual=x)
    ops.distill_loss(ops.linear(y, w["out.weight"]), t, index, temperature=2.0).sum().backward()
    for k, v in w.items():
        assert torch.equal(v.grad, grads[k]), k
