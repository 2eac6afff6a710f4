"""Activations at pre-activations whose square or cube leaves fp32's range."""
import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_large_preactivations(act):
    from tensor_grad_clip_gb300 import ops
    big = torch.tensor([1e10, 1e13, 1e18, 1e19, 1e20, 3e25, 1e30, 3e38], device="cuda").bfloat16()
    z = torch.cat([big, -big, torch.linspace(-100, 100, 48, device="cuda").bfloat16()])[None].expand(20, 64).contiguous()
    n = z.shape[1]
    one = torch.eye(n, device="cuda", dtype=torch.bfloat16)
    # forward: the product is z itself
    y = ops.linear_forward(z, one, activation=act)
    want = torch.where(z.double().abs() > 1e3, z.double() * (1.0 if act == "none" else z > 0), R.activate(z.double(), act))
    R.assert_close(y, want, R.rounding(want, torch.bfloat16) + 1e-6 * z.double().abs().clamp(max=1e3), "y")
    # backward with dy = 1: dx is the slope, 0 or 1 far out
    dy = torch.ones_like(z)
    dx, _, db = ops.linear_backward(dy, z, one, z, activation=act, weight_grad=False)
    far = z.double().abs() > 1e3
    want = torch.ones_like(z.double()) if act == "none" else torch.where(far, (z > 0).double(),
                                                                         R.act_slope(z.double().clamp(-1e3, 1e3), act))
    R.assert_close(dx, want, 2 * R.rounding(want, torch.bfloat16) + 1e-5, "dx")
    R.assert_close(db, want.sum(0), R.rounding(want.sum(0), torch.bfloat16) + 20e-5, "dbias")
