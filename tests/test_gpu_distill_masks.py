"""Distillation loss where logits are masked: what the contract says of -inf, of a row that is wholly masked, and of the
type's lowest value, which is an ordinary logit."""
import math

import pytest
import torch

import ops_reference as R
from test_gpu_distill import DT, LOWEST, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def against_fp64(ops, z, t, index, w, g, T):
    loss, lse = ops.distill_forward(z, t, index, temperature=T, row_weight=w)
    rloss, rlse, rd = R.distill(z, t, index, T, w)
    tloss, tlse, td = R.distill_bounds(z, t, index, T, w)
    R.assert_close(lse, rlse, tlse, "lse")
    R.assert_close(loss, rloss, tloss, "loss")
    loss2, d = ops.distill_loss_grad(z, t, index, temperature=T, row_weight=w)
    R.assert_close(loss2, rloss, tloss, "loss of loss_grad")
    R.assert_close(d, rd, td + R.rounding(rd, z.dtype), "dlogits of loss_grad")
    rd, td = R.distill(z, t, index, T, w, g)[2], R.distill_bounds(z, t, index, T, w, g)[2]
    d2 = ops.distill_backward(g, z, lse, t, index, temperature=T, row_weight=w)
    R.assert_close(d2, rd, td + R.rounding(rd, z.dtype), "dlogits")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,vocab", [(4, 500), (3, 40001), (620, 17000)])
def test_the_lowest_value_at_a_teachers_entry(ops, dtype, rows, vocab):
    z, t, index, w, g = problem(rows, vocab, 6, dtype)
    z[1].scatter_(0, index[1, :2].long(), LOWEST[dtype])
    z[2] = LOWEST[dtype]
    z[2, index[2, 0].long()] = 1.0
    against_fp64(ops, z, t, index, w, g, 1.0)
    if dtype == torch.float16:  # 65504 / 5000: q is not 0 there
        against_fp64(ops, z, t, index, w, g, 5000.0)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,vocab", [(6, 500), (5, 40001), (700, 17000)])
def test_rows_wholly_masked(ops, dtype, rows, vocab):
    z, t, index, w, g = problem(rows, vocab, 6, dtype)
    clean, clean_lse = ops.distill_forward(z, t, index, row_weight=w)
    clean_d = ops.distill_loss_grad(z, t, index, row_weight=w)[1]
    z[1] = z[2] = z[3] = -math.inf
    index[2] = -1
    w[3] = 0
    loss, lse = ops.distill_forward(z, t, index, row_weight=w)
    loss2, d = ops.distill_loss_grad(z, t, index, row_weight=w)
    d2 = ops.distill_backward(g, z, lse, t, index, row_weight=w)
    for v in (loss, loss2):
        assert torch.isnan(v[1]) and v[2] == 0 and v[3] == 0
    assert lse[1] == -math.inf and lse[2] == -math.inf and lse[3] == 0
    for v in (d, d2):
        assert torch.isnan(v[1]).all() and not v[2].any() and not v[3].any()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[1:4] = False
    assert torch.equal(loss[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    assert torch.equal(d[keep], clean_d[keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_beyond_fp32_at_their_temperature(ops, dtype):
    z, t, index, w, g = problem(4, 900, 6, dtype)
    z[1, 100:] = LOWEST[dtype]  # z / T is -inf: as if masked with it
    z[1].scatter_(0, index[1].long(), 1.0)
    masked = z.clone()
    masked[1][z[1] == LOWEST[dtype]] = -math.inf
    for a, b in zip(ops.distill_loss_grad(z, t, index, temperature=0.25),
                    ops.distill_loss_grad(masked, t, index, temperature=0.25)):
        assert torch.equal(a, b) and torch.isfinite(a).all()
