"""What the training operators' calls promise beside their values: the device check waits, rows that do not count, outputs
that autograd knows of, nothing stored that nobody reads."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def test_check_waits_for_other_streams(ops):
    x = torch.randn(64, 512, device="cuda")
    ops.layer_norm_forward(x)
    ops.check(0)  # (loads what the check itself needs)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
        ops.layer_norm_forward(x)
        last = torch.cuda.Event()
        last.record()
    assert not last.query()
    ops.check(0)
    assert last.query()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_row_of_weight_0_whatever_its_loss_gradient(ops, bad):
    for vocab, dtype in ((500, torch.float32), (40001, torch.bfloat16), (40000, torch.float16)):
        z = torch.randn(5, vocab, device="cuda").to(dtype)
        t, index = torch.randn(5, 6, device="cuda"), torch.randint(0, vocab, (5, 6), device="cuda")
        w, g = torch.ones(5, device="cuda"), torch.ones(5, device="cuda")
        _, lse = ops.distill_forward(z, t, index)
        clean = ops.distill_backward(g, z, lse, t, index, row_weight=w)
        w[1], g[1], z[1] = 0, bad, math.nan
        w[3], g[3] = 0, bad
        d = ops.distill_backward(g, z, lse, t, index, row_weight=w)
        assert not d[1].any() and not d[3].any()
        for r in (0, 2, 4):
            assert torch.equal(d[r], clean[r])


def test_autograd_knows_of_logits_that_a_gradient_replaced(ops):
    t, index = torch.randn(4, 6, device="cuda"), torch.randint(0, 300, (4, 6), device="cuda")
    for call in ("loss_grad", "backward"):
        z = torch.randn(4, 300, device="cuda", requires_grad=True)
        loss = ops.distill_loss(z, t, index)
        place = z.detach()  # the same memory
        if call == "loss_grad":
            ops.distill_loss_grad(place, t, index, out=place)
        else:
            ops.distill_backward(torch.ones(4, device="cuda"), place, ops.distill_forward(place, t, index)[1], t, index,
                                 out=place)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.sum().backward()
    with torch.inference_mode():  # (such tensors have no version)
        z = torch.randn(4, 300, device="cuda")
        want = ops.distill_loss_grad(z, t, index)[1]
        assert torch.equal(ops.distill_loss_grad(z, t, index, out=z)[1], want)


def test_no_preactivation_is_stored_without_a_gradient(ops, monkeypatch):
    asked = []
    real = ops.linear_forward

    def spy(*args, **kwargs):
        asked.append(kwargs.get("save_preactivation", False))
        return real(*args, **kwargs)
    monkeypatch.setattr(ops, "linear_forward", spy)
    x, w, r = (torch.randn(s, device="cuda").half() for s in ((20, 64), (48, 64), (20, 48)))
    want = real(x, w, activation="gelu", residual=r)
    wg = w.clone().requires_grad_()
    with torch.no_grad():
        assert torch.equal(ops.linear(x, wg, activation="gelu", residual=r), want)
    assert torch.equal(ops.linear(x, w, activation="gelu", residual=r), want)
    rg = r.clone().requires_grad_()
    y = ops.linear(x, w, activation="gelu", residual=rg)  # the residual's gradient is dy itself
    y.backward(torch.ones_like(y))
    assert torch.equal(y, want) and torch.equal(rg.grad, torch.ones_like(r))
    assert asked == [False, False, False]
    y = ops.linear(x, wg, activation="gelu", residual=r)
    y.backward(torch.ones_like(y))
    assert torch.equal(y, want) and asked[3:] == [True]
    z = real(x, w, activation="gelu", save_preactivation=True)[1]
    assert torch.equal(wg.grad, ops.linear_backward(torch.ones_like(y), x, w, z, activation="gelu")[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_bits_wherever_rows_start(ops, dtype):
    for rows, cols in ((9, 500), (300, 4099), (20, 16384)):
        flat = torch.randn(rows, cols, device="cuda").to(dtype)
        w = torch.rand(cols, device="cuda")

        def norm(x):
            y, mu, rstd = ops.layer_norm_forward(x, w, w)
            return y, mu, rstd, *ops.layer_norm_backward(x, x, w, mu, rstd)
        for other in moved(flat):
            assert all(torch.equal(a, b) for a, b in zip(norm(flat), norm(other)))
    for rows, vocab in ((3, 40000), (100, 9000), (700, 17000)):
        z = torch.randn(rows, vocab, device="cuda").mul(2.5).to(dtype)
        t, index = torch.randn(rows, 9, device="cuda"), torch.randint(0, vocab, (rows, 9), device="cuda")
        g = torch.randn(rows, device="cuda")

        def distill(z):
            loss, lse = ops.distill_forward(z, t, index)
            # (loss and gradient together too, except of many long rows: these go through shared memory where they are aligned)
            return loss, lse, ops.distill_backward(g, z, lse, t, index), *(
                ops.distill_loss_grad(z, t, index) if rows < 600 else ())
        for other in moved(z):
            assert all(torch.equal(a, b) for a, b in zip(distill(z), distill(other)))


def moved(x):
    """x's values in rows that start elsewhere."""
    rows, cols = x.shape
    for pad, offset in ((0, 3), (3, 1), (8, 0)):
        buf = torch.zeros(rows * (cols + pad) + offset, device="cuda", dtype=x.dtype)
        view = buf[offset:].view(rows, cols + pad)[:, :cols]
        view.copy_(x)
        yield view
