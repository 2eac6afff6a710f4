"""Host side of the language model operators' C ABI: bad arguments are refused with a status and a text before anything
reaches the GPU (every call here is invalid in at least one respect, or has nothing to compute)."""
import ctypes

import pytest
import torch

from tensor_grad_clip_gb300 import _abi, _ops_abi as C, build

P = 1 << 20  # a pointer that is aligned and never followed


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return C.load()


def text():
    return C.soma_ops_last_error().decode()


def lookup(w=P, ws=64, i=P, ins=8, batch=2, length=8, y=P, ys=64, vocab=100, cols=64, dt=1, it=1, scale=1.0):
    return C.soma_embedding_forward(0, w, ws, i, ins, batch, length, y, ys, vocab, cols, dt, it, scale, None)


def gradient(dy=P, dys=64, i=P, ins=8, batch=2, length=8, dw=P, dws=64, acc=0, ws=P, nbytes=1 << 30, vocab=100, cols=64,
             dt=1, it=1, scale=1.0):
    return C.soma_embedding_backward(0, dy, dys, i, ins, batch, length, dw, dws, acc, ws, nbytes, vocab, cols, dt, it,
                                     scale, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(batch=-1), 1, "batch"), (dict(length=-1), 1, "batch"), (dict(batch=1 << 20, length=1 << 11), 1, "batch"),
    (dict(batch=1 << 62, length=4), 1, "batch"), (dict(vocab=0), 1, "vocab"), (dict(vocab=(1 << 30) + 1), 1, "vocab"),
    (dict(cols=0), 1, "cols"), (dict(cols=(1 << 30) + 1), 1, "cols"), (dict(dt=3), _abi.SOMA_ERR_DTYPE, "dtype"),
    (dict(it=2), _abi.SOMA_ERR_DTYPE, "index_type"), (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=1e39), 1, "scale"), (dict(i=None), 1, "index is NULL"), (dict(i=P + 4), _abi.SOMA_ERR_ALIGNMENT, "index"),
    (dict(ins=7), 1, "index: stride"),
])
def test_embedding_refusals(kw, status, word):
    for call in (lookup, gradient):
        assert call(**kw) == status
        assert word in text()


def test_embedding_buffers():
    for call, kw, status, word in (
            (lookup, dict(w=None), 1, "weight is NULL"), (lookup, dict(ws=63), 1, "weight: stride"),
            (lookup, dict(y=None), 1, "y is NULL"), (lookup, dict(ys=-1), 1, "y: stride"), (lookup, dict(y=P + 1), 4, "y"),
            (lookup, dict(w=P + 2, dt=0), 4, "weight"), (gradient, dict(dy=None), 1, "dy is NULL"),
            (gradient, dict(dys=63), 1, "dy: stride"), (gradient, dict(dw=None), 1, "dweight is NULL"),
            (gradient, dict(dws=63), 1, "dweight: stride"), (gradient, dict(dw=P + 1), 4, "dweight"),
            (gradient, dict(acc=2), 1, "accumulate"), (gradient, dict(ws=None), 1, "workspace is NULL"),
            (gradient, dict(nbytes=100), _abi.SOMA_ERR_LIMIT, "workspace has"),
            (gradient, dict(ws=P + 64), 4, "workspace is not")):
        assert call(**kw) == status and word in text(), kw


def test_embedding_workspace():
    need = ctypes.c_int64(7)
    assert C.soma_embedding_backward_workspace(0, 4, 10, 8, None) == 1
    for rows, vocab, cols in ((-1, 10, 8), (1 << 31, 10, 8), (4, 0, 8), (4, 10, 0)):
        assert C.soma_embedding_backward_workspace(0, rows, vocab, cols, ctypes.byref(need)) == 1
    assert need.value == 7
    assert C.soma_embedding_backward_workspace(0, 0, 10, 8, ctypes.byref(need)) == 0 and need.value == 0
    assert C.soma_embedding_backward_workspace(0, 4, 10, 8, ctypes.byref(need)) == 0 and need.value >= 2 * 4 * 4


def test_nothing_to_compute_succeeds():
    assert lookup(batch=0, i=None, y=None) == 0 and lookup(length=0, i=None, y=None) == 0
    assert gradient(batch=0, i=None, dy=None, acc=1, ws=None, nbytes=0) == 0


def test_python_refuses_host_tensors():
    from tensor_grad_clip_gb300 import ops
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ops.embedding_forward(i, x), lambda: ops.embedding_backward(x, i, 10)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a process without a GPU")
def test_without_a_gpu_a_valid_call_reports_cuda():
    assert lookup() == _abi.SOMA_ERR_CUDA and gradient() == _abi.SOMA_ERR_CUDA


# ---- cross entropy of a linear layer ------------------------------------------

def head(x=P, xs=64, w=P, ws=64, t=P, ts=8, batch=2, length=8, rw=P, loss=P, lse=P, work=P, nbytes=1 << 40, vocab=100, k=64,
         dt=1, it=1):
    return C.soma_linear_cross_entropy_forward(0, x, xs, w, ws, t, ts, batch, length, rw, loss, lse, work, nbytes, vocab, k,
                                               dt, it, None)


def head_backward(g=P, x=P, xs=64, w=P, ws=64, t=P, ts=8, batch=2, length=8, rw=P, lse=P, dx=P, dxs=64, dw=P, dws=64, work=P,
                  nbytes=1 << 40, vocab=100, k=64, dt=1, it=1):
    return C.soma_linear_cross_entropy_backward(0, g, x, xs, w, ws, t, ts, batch, length, lse, rw, dx, dxs, dw, dws, work,
                                                nbytes, vocab, k, dt, it, None)


def head_both(x=P, xs=64, w=P, ws=64, t=P, ts=8, batch=2, length=8, rw=P, loss=P, lse=P, dx=P, dxs=64, dw=P, dws=64, work=P,
              nbytes=1 << 40, vocab=100, k=64, dt=1, it=1):
    return C.soma_linear_cross_entropy_loss_grad(0, x, xs, w, ws, t, ts, batch, length, rw, loss, lse, dx, dxs, dw, dws, work,
                                                 nbytes, vocab, k, dt, it, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(batch=-1), 1, "batch"), (dict(length=-1), 1, "batch"), (dict(batch=1 << 40, length=1 << 40), 1, "batch"),
    (dict(batch=(1 << 30) + 1, length=1, ts=1), 1, "2^30"), (dict(vocab=0), 1, "vocab"),
    (dict(vocab=(1 << 30) + 1), 1, "vocab"), (dict(k=0), 1, "k must"), (dict(k=1 << 31), 1, "k must"),
    (dict(dt=0), _abi.SOMA_ERR_DTYPE, "bf16 or fp16"), (dict(it=7), _abi.SOMA_ERR_DTYPE, "index_type"),
    (dict(x=None), 1, "x is NULL"), (dict(xs=63), 1, "x: stride"), (dict(x=P + 1), 4, "x"),
    (dict(w=None), 1, "weight is NULL"), (dict(ws=63), 1, "weight: stride"), (dict(w=P + 1), 4, "weight"),
    (dict(t=None), 1, "target is NULL"), (dict(ts=7), 1, "target: stride"), (dict(t=P + 4), 4, "target"),
    (dict(rw=P + 2), 4, "row_weight"),
])
def test_head_refusals(kw, status, word):
    for call in (head, head_backward, head_both):
        assert call(**kw) == status
        assert word in text()


def test_head_buffers():
    for call, kw, status, word in (
            (head, dict(loss=P + 1), 4, "loss"), (head, dict(lse=P + 2), 4, "lse"), (head_both, dict(loss=None), 1, "loss"),
            (head_both, dict(dx=P + 1), 4, "dx"), (head_both, dict(dxs=63), 1, "dx: stride"),
            (head_both, dict(dw=P + 1), 4, "dweight"), (head_both, dict(dws=63), 1, "dweight: stride"),
            (head_backward, dict(g=None), 1, "grad_loss"), (head_backward, dict(lse=None), 1, "lse"),
            (head_backward, dict(g=P + 2), 4, "grad_loss")):
        assert call(**kw) == status and word in text(), kw
    need = ctypes.c_int64()
    assert C.soma_linear_cross_entropy_workspace(0, P, 64, 16, 100, 64, 1, 1, 1, 1, None) == 1
    for rows, vocab, k, dt in ((-1, 100, 64, 1), ((1 << 30) + 1, 100, 64, 1), (16, 0, 64, 1), (16, 100, 0, 1), (16, 100, 64, 0)):
        assert C.soma_linear_cross_entropy_workspace(0, P, 64, rows, vocab, k, dt, 1, 1, 1, ctypes.byref(need)) != 0


def test_head_with_nothing_to_compute():
    assert head(batch=0, x=None, t=None, loss=None, lse=None) == 0
    assert head_backward(dx=None, dw=None) == 0
    assert head_both(length=0, x=None, t=None, loss=None, dx=None, dw=None) == 0


def test_head_python_refuses_host_tensors():
    from tensor_grad_clip_gb300 import ops
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.linear_cross_entropy_forward(x, x, torch.zeros(4, dtype=torch.int64))


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a process without a GPU")
def test_head_without_a_gpu_reports_cuda():
    assert head() == _abi.SOMA_ERR_CUDA and head_backward() == _abi.SOMA_ERR_CUDA and head_both() == _abi.SOMA_ERR_CUDA
