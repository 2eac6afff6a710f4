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
