"""Layer norm where fp32 loses bits easily, against its formulas in fp64: large channels in the middle of a row, rows
whose mean is far from 0, and row lengths at the limit."""
import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def check_forward(ops, x):
    y, mu, rstd = ops.layer_norm_forward(x)
    ry, rmu, rrstd = R.norm_forward(x, None, None, 1e-5)
    ty, tmu, trstd = R.norm_forward_bounds(x, None, None, 1e-5, ry, rmu, rrstd)
    R.assert_close(mu, rmu, tmu, "mean")
    R.assert_close(rstd, rrstd, trstd, "rstd")
    R.assert_close(y, ry, ty + R.rounding(ry, x.dtype), "y")


@pytest.mark.parametrize("cols,pad", [(7, 0), (100, 0), (500, 0), (500, 1), (1000, 0), (4096, 0), (4099, 0), (8192, 0),
                                      (16384, 0), (16384, 3), (20000, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_large_channels_in_the_middle(ops, cols, pad, dtype):
    for rows, size in ((3, 1e4), (400, 300.0), (400, 1e4)):
        gen = torch.Generator(device="cuda").manual_seed(cols + rows)
        x = torch.randn(rows, cols + pad, device="cuda", generator=gen)[:, :cols].to(dtype)
        for shift in range(8):  # row r's channel sits r % 8 places before or after the middle
            x[shift::8, max(0, min(cols - 1, cols // 2 + shift - 4))] = size if shift % 2 else -size
        x[1, cols // 2 - 2:cols // 2 + 3] = size  # several of them
        check_forward(ops, x)
        check_forward(ops, x + 50)


@pytest.mark.parametrize("cols", [300, 1000, 4096, 4099, 16384, 20000])
@pytest.mark.parametrize("dtype,mean", [(torch.float32, 1e3), (torch.float32, 1e4), (torch.bfloat16, 100.0)])
def test_gradient_of_rows_far_from_zero(ops, cols, dtype, mean):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn(37, cols, device="cuda", generator=gen) + mean).to(dtype)
    w = torch.rand(cols, device="cuda", generator=gen) + 0.5
    _, mu, rstd = ops.layer_norm_forward(x, w)
    xh = (x.double() - mu.double()[:, None]) * rstd.double()[:, None]
    dy = (xh + torch.randn(37, cols, device="cuda", generator=gen)).to(dtype)  # mean(g xh) is about 1
    dx, dw, db = ops.layer_norm_backward(dy, x, w, mu, rstd)
    rdx, rdw, rdb = R.norm_backward(dy, x, w, mu, rstd)
    # x - mean rounds to 2^-24 of itself and so does its product with rstd: the errors of xh go with |xh|, not with
    # |x| + |mean| (centred x and a mean of 0 give such bounds)
    tdx, tdw, _ = R.norm_backward_bounds(dy, x.double() - mu.double()[:, None], w, torch.zeros_like(mu), rstd)
    R.assert_close(dx, rdx, tdx + R.rounding(rdx, dtype), "dx")
    R.assert_close(dw, rdw, tdw + R.rounding(rdw, torch.float32), "dweight")


def test_the_longest_row(ops):
    cols = 2 ** 31 - 1
    x = torch.empty(0, cols, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(cols, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, device="cuda")
    _, dw, db = ops.layer_norm_backward(x, x, w, none, none)
    assert dw.shape == db.shape == (cols,)
    assert not dw.view(torch.int16).any() and not db.view(torch.int16).any()
    del x, w, dw, db
    torch.cuda.empty_cache()
