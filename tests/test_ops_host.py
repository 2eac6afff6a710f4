"""Host side of the training operators' C ABI: every function that
include/soma_ops.h declares is exported and bound, and bad arguments are
refused with a status and a text before anything reaches the GPU (every call
here is invalid in at least one respect, or has nothing to compute)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from tensor_grad_clip_gb300 import _abi, _ops_abi as C, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a pointer that is aligned and never followed


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return C.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "soma_ops.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(soma_\w+)\s*\(", text))
    assert names == set(C.SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_is_c99(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "soma_ops.h"\nint main(void) { return SOMA_ACT_NONE; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)


def text():
    return C.soma_ops_last_error().decode()


def norm(x=P, xs=64, w=P, b=P, y=P, ys=64, mu=P, rstd=P, rows=4, cols=64, dt=1, pdt=0, eps=1e-5):
    return C.soma_layer_norm_forward(0, x, xs, w, b, y, ys, mu, rstd, rows, cols, dt, pdt, eps, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), _abi.SOMA_ERR_INVALID_ARG, "rows"),
    (dict(cols=0), _abi.SOMA_ERR_INVALID_ARG, "cols"),
    (dict(cols=1 << 31, xs=1 << 31, ys=1 << 31), _abi.SOMA_ERR_INVALID_ARG, "cols"),
    (dict(dt=3), _abi.SOMA_ERR_DTYPE, "dtype"),
    (dict(dt=1, pdt=2), _abi.SOMA_ERR_DTYPE, "param_dtype"),
    (dict(eps=-1e-9), _abi.SOMA_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), _abi.SOMA_ERR_INVALID_ARG, "eps"),
    (dict(x=None), _abi.SOMA_ERR_INVALID_ARG, "x is NULL"),
    (dict(y=None), _abi.SOMA_ERR_INVALID_ARG, "y is NULL"),
    (dict(xs=63), _abi.SOMA_ERR_INVALID_ARG, "stride"),
    (dict(ys=-64), _abi.SOMA_ERR_INVALID_ARG, "stride"),
    (dict(xs=1 << 61), _abi.SOMA_ERR_LIMIT, "64 bits"),
    (dict(x=P + 1), _abi.SOMA_ERR_ALIGNMENT, "x"),
    (dict(w=P + 2), _abi.SOMA_ERR_ALIGNMENT, "weight"),
    (dict(mu=P + 2), _abi.SOMA_ERR_ALIGNMENT, "mean"),
])
def test_layer_norm_refusals(kw, status, word):
    assert norm(**kw) == status
    assert word in text()


def test_nothing_to_compute_succeeds():
    assert norm(rows=0, x=None, y=None, mu=None, rstd=None) == 0
    assert C.soma_layer_norm_backward(0, None, 64, None, 64, None, None, None, None, 64, None, None, None, 0, 0, 64,
                                      0, 0, None) == 0
    assert linear(m=0, x=None, y=None) == 0
    assert linear(n=0, w=None, y=None, b=None) == 0
    assert distill(rows=0, z=None, t=None, i=None, loss=None, lse=None) == 0


def test_layer_norm_backward_refusals():
    def call(dy=P, x=P, w=P, mu=P, rstd=P, dx=P, dw=None, db=None, stride=64):
        return C.soma_layer_norm_backward(0, dy, stride, x, stride, w, mu, rstd, dx, stride, dw, db, None, 0, 4, 64,
                                          0, 0, None)
    for kw, status, word in ((dict(dy=None), 1, "dy"), (dict(x=None), 1, "x"), (dict(mu=None), 1, "mean"),
                             (dict(rstd=None), 1, "rstd"), (dict(dx=P + 2), 4, "dx"), (dict(dw=P + 1), 4, "dweight"),
                             (dict(db=P + 3), 4, "dbias"), (dict(stride=60), 1, "stride")):
        assert call(**kw) == status and word in text(), kw
    assert C.soma_layer_norm_backward_workspace(0, 4, 64, None) == 1


def linear(x=P, xs=32, w=P, ws=32, b=P, r=None, rs=48, y=P, ys=48, z=None, zs=48, m=4, n=48, k=32, dt=1, act=0):
    return C.soma_linear_forward(0, x, xs, w, ws, b, r, rs, y, ys, z, zs, None, 0, m, n, k, dt, act, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(m=-1), 1, "m and n"), (dict(n=1 << 31), 1, "m and n"), (dict(k=0), 1, "k must"),
    (dict(dt=0), _abi.SOMA_ERR_DTYPE, "bf16 or fp16"), (dict(act=5), 1, "activation"), (dict(act=-1), 1, "activation"),
    (dict(x=None), 1, "x is NULL"), (dict(w=None), 1, "weight is NULL"), (dict(y=None), 1, "y is NULL"),
    (dict(xs=31), 1, "stride"), (dict(ws=-32), 1, "stride"), (dict(ys=47), 1, "stride"),
    (dict(r=P, rs=47), 1, "residual"), (dict(z=P, zs=40), 1, "z_out"), (dict(b=P + 1), 4, "bias"),
    (dict(x=P + 1), 4, "x"),
])
def test_linear_refusals(kw, status, word):
    assert linear(**kw) == status
    assert word in text()


def test_linear_backward_refusals():
    def call(dy=P, x=P, w=P, z=P, dx=P, dw=P, db=P, m=4, n=48, k=32, dt=1, act=1, dys=48):
        return C.soma_linear_backward(0, dy, dys, x, 32, w, 32, z, 48, dx, 32, dw, 32, db, None, 0, m, n, k, dt, act,
                                      None)
    for kw, status, word in ((dict(dy=None), 1, "dy"), (dict(x=None), 1, "x is NULL"), (dict(w=None), 1, "weight"),
                             (dict(z=None), 1, "z is NULL"), (dict(dys=47), 1, "dy"), (dict(dt=0), 3, "bf16"),
                             (dict(k=0), 1, "k must"), (dict(dx=P + 1), 4, "dx"), (dict(dw=P + 1), 4, "dweight"),
                             (dict(db=P + 1), 4, "dbias"), (dict(act=7), 1, "activation")):
        assert call(**kw) == status and word in text(), kw
    assert C.soma_linear_backward_workspace(0, P, 48, P, 32, P, 32, 4, 48, 32, 1, 1, None) == 1
    assert C.soma_linear_forward_workspace(0, P, 32, P, 32, 4, 48, 32, 1, None) == 1


def distill(z=P, zs=100, t=P, ts=8, i=P, ins=8, w=P, T=1.0, loss=P, lse=P, rows=4, vocab=100, top=8, dt=0, tdt=0,
            it=0):
    return C.soma_distill_forward(0, z, zs, t, ts, i, ins, w, T, loss, lse, rows, vocab, top, dt, tdt, it, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), 1, "rows"), (dict(vocab=0), 1, "vocab"), (dict(vocab=1 << 31), 1, "vocab"),
    (dict(top=-1), 1, "top"), (dict(top=1025, ts=1025, ins=1025), _abi.SOMA_ERR_LIMIT, "top"),
    (dict(dt=3), 3, "dtype"), (dict(tdt=-1), 3, "teacher_dtype"), (dict(it=2), 3, "index_type"),
    (dict(T=0.0), 1, "temperature"), (dict(T=-1.0), 1, "temperature"), (dict(T=float("nan")), 1, "temperature"),
    (dict(T=float("inf")), 1, "temperature"), (dict(z=None), 1, "logits"), (dict(t=None), 1, "teacher"),
    (dict(i=None), 1, "index"), (dict(loss=None), 1, "loss"), (dict(lse=None), 1, "lse"), (dict(zs=99), 1, "stride"),
    (dict(z=P + 2), 4, "logits"), (dict(i=P + 4, it=1), 4, "index"), (dict(w=P + 1), 4, "row_weight"),
])
def test_distill_refusals(kw, status, word):
    assert distill(**kw) == status
    assert word in text()


def test_distill_gradient_refusals():
    def backward(g=P, lse=P, d=P, ds=100):
        return C.soma_distill_backward(0, g, P, 100, lse, P, 8, P, 8, None, 1.0, d, ds, 4, 100, 8, 0, 0, 0, None)
    for kw, word in ((dict(g=None), "grad_loss"), (dict(lse=None), "lse"), (dict(d=None), "dlogits"),
                     (dict(ds=99), "stride")):
        assert backward(**kw) == 1 and word in text(), kw
    assert C.soma_distill_loss_grad(0, P, 100, P, 8, P, 8, None, 1.0, P, None, None, 100, 4, 100, 8, 0, 0, 0,
                                    None) == 1 and "dlogits" in text()


def test_python_refuses_host_tensors():
    from tensor_grad_clip_gb300 import ops
    x = torch.zeros(4, 8)
    for call in (lambda: ops.layer_norm_forward(x), lambda: ops.linear_forward(x, x),
                 lambda: ops.distill_forward(x, x, x.int())):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a process without a GPU")
def test_without_a_gpu_a_valid_call_reports_cuda():
    assert norm() == _abi.SOMA_ERR_CUDA
    need = ctypes.c_int64()
    assert C.soma_layer_norm_backward_workspace(0, 4, 64, ctypes.byref(need)) == _abi.SOMA_ERR_CUDA
