"""The kernels' bounded waits: limits that leave long sums their time (checked by the compiler, here), and on a GPU what a
wait does whose barrier nothing arrives at, and the longest sum of products that is worth a test."""
import ctypes
import os
import subprocess

import pytest
import torch

from tensor_grad_clip_gb300 import build

PROBE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "wait_probe.cu")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("probe") / "wait_probe.so")
    subprocess.run([build.nvcc(), "-std=c++17", "-O3", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
                    "-I", build.CSRC, "-I", build.INCLUDE, *build.ARCH, PROBE, "-o", lib], check=True)
    return ctypes.CDLL(lib)


def test_limits(probe):
    assert probe.run_probe


def run(probe, arrives, limit):
    out = (ctypes.c_longlong * 4)()
    assert probe.run_probe(arrives, ctypes.c_ulonglong(limit), out) == 0
    return list(out)


@pytest.mark.gpu
def test_a_wait_ends(probe):
    assert run(probe, 1, 10 ** 9)[:2] == [1, 1]
    mine, other, mine_ns, other_ns = run(probe, 0, 20_000_000)  # 20 ms
    assert (mine, other) == (0, 0)
    assert 20_000_000 <= mine_ns < 500_000_000 and other_ns < 500_000_000
    assert run(probe, 1, 10 ** 9)[:2] == [1, 1]


@pytest.mark.gpu
def test_a_long_sum():
    from tensor_grad_clip_gb300 import ops
    rows = 2 ** 28  # 4 M pipeline stages over eight CTAs; every partial sum of ones is exact
    x = torch.ones(rows, 64, device="cuda", dtype=torch.bfloat16)
    dy = torch.ones(rows, 8, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(8, 64, device="cuda", dtype=torch.bfloat16)
    _, dw, _ = ops.linear_backward(dy, x, w, input_grad=False, bias_grad=False)
    assert (dw == 2 ** 28).all()
    ops.check(0)
    del x, dy, dw
    torch.cuda.empty_cache()
