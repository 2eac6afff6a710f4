"""The training operators where element offsets pass 32 bits: the last rows
of matrices of more than 2^31 elements against fp64, and the device check."""
import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def rows_at_the_end(x, n=3):
    return x[-n:].clone()


def test_layer_norm(ops):
    rows, cols = 530000, 4099  # 2.17e9 elements, rows at every alignment
    x = torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16)
    w, b = torch.rand(cols, device="cuda"), torch.rand(cols, device="cuda")
    y, mu, rstd = ops.layer_norm_forward(x, w, b)
    xe = rows_at_the_end(x)
    ry, rmu, rrstd = R.norm_forward(xe, w, b, 1e-5)
    ty, tmu, _ = R.norm_forward_bounds(xe, w, b, 1e-5, ry, rmu, rrstd)
    R.assert_close(y[-3:], ry, ty + R.rounding(ry, x.dtype), "y")
    R.assert_close(mu[-3:], rmu, tmu, "mean")
    dx, _, db = ops.layer_norm_backward(y, x, w, mu, rstd)
    rdx, _, _ = R.norm_backward(y[-3:], xe, w, mu[-3:], rstd[-3:])
    tdx, _, _ = R.norm_backward_bounds(y[-3:], xe, w, mu[-3:], rstd[-3:])
    R.assert_close(dx[-3:], rdx, tdx + R.rounding(rdx, x.dtype), "dx")
    assert torch.isfinite(db).all()


def test_linear(ops):
    m, n, k = 66000, 32768, 64  # 2.16e9 outputs
    x, w = torch.randn(m, k, device="cuda").bfloat16(), torch.randn(n, k, device="cuda").bfloat16()
    y = ops.linear_forward(x, w)
    ry, _ = R.linear_forward(x[-3:], w, None, "none", None)
    ty, _ = R.linear_forward_bounds(x[-3:], w, None, "none", None)
    R.assert_close(y[-3:], ry, ty + R.rounding(ry, x.dtype), "y")
    dx, dw, db = ops.linear_backward(y, x, w, y, activation="relu")
    rdx, _, _ = R.linear_backward(y[-3:], x[-3:], w, y[-3:], "relu")
    tdx, _, _ = R.linear_backward_bounds(y[-3:], x[-3:], w, y[-3:], "relu", x.dtype)
    R.assert_close(dx[-3:], rdx, tdx + R.rounding(rdx, x.dtype), "dx")
    assert torch.isfinite(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("vocab", [32768, 32771])
def test_distillation(ops, vocab):
    rows = 66000
    z = torch.randn(rows, vocab, device="cuda", dtype=torch.bfloat16)
    index = (torch.arange(8, device="cuda") * 4001 + torch.randint(0, 4001, (rows, 8), device="cuda")).int()
    t = torch.randn(rows, 8, device="cuda") + 3
    loss, lse = ops.distill_forward(z, t, index)
    rloss, rlse, rd = R.distill(z[-3:], t[-3:], index[-3:], 1.0)
    tloss, tlse, td = R.distill_bounds(z[-3:], t[-3:], index[-3:], 1.0)
    R.assert_close(loss[-3:], rloss, tloss, "loss")
    R.assert_close(lse[-3:], rlse, tlse, "lse")
    d = ops.distill_backward(torch.ones_like(loss), z, lse, t, index)
    R.assert_close(d[-3:], rd, td + R.rounding(rd, z.dtype), "dlogits")
    loss, d = ops.distill_loss_grad(z, t, index, out=z)
    R.assert_close(loss[-3:], rloss, tloss, "loss of loss_grad")
    R.assert_close(d[-3:], rd, td + R.rounding(rd, z.dtype), "dlogits of loss_grad")


def test_no_kernel_gave_up(ops):
    ops.check(0)
