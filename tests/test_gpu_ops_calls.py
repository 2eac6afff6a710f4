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
