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
