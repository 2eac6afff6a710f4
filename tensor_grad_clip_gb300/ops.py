"""Training operators whose gradients the optimizer step takes: layer norm,
linear layer, distillation loss, embedding and the cross entropy of a linear
layer over a vocabulary, each forward and backward, as sm_103a kernels behind
the C ABI of include/soma_ops.h (formulas there).

Explicit calls, for programs that keep their own backward pass::

    y, mean, rstd = layer_norm_forward(x, weight, bias)
    h, z = linear_forward(y, w1, b1, activation="gelu", save_preactivation=True)
    logits = linear_forward(h, w2)
    loss, dlogits = distill_loss_grad(logits, teacher_logits, teacher_index, temperature=2.0)
    dh, dw2, _ = linear_backward(dlogits, h, w2, bias_grad=False)
    dy, dw1, db1 = linear_backward(dh, y, w1, z, activation="gelu")
    dx, dweight, dbias = layer_norm_backward(dy, x, weight, mean, rstd)

and for a language model's two ends, here with one table for both::

    x = embedding_forward(tokens, table)
    loss, dy, dtable = linear_cross_entropy_loss_grad(y, table, targets)
    embedding_backward(dx, tokens, len(table), out=dtable)

and the same with autograd: layer_norm, linear, distill_loss, embedding,
linear_cross_entropy.

Tensors are CUDA tensors with unit stride in the last dimension; all leading
dimensions are rows and must be evenly spaced (any tensor that can be viewed
as [rows, last]).  Tokens may be a slice tokens[:, 1:] or a column tokens[:, -1]
of a batch of texts.  Work is enqueued on the current stream, or on `stream` (a
torch stream or a raw cudaStream_t), which then also owns the outputs; the
inputs are kept alive for it.  Nothing waits for the GPU, and there is no
fallback: a refused call raises SomaError, ValueError or TypeError.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import SomaError, _ops_abi
from ._abi import SOMA_DTYPE_BF16, SOMA_DTYPE_F16, SOMA_DTYPE_F32

__all__ = ["layer_norm_forward", "layer_norm_backward", "linear_forward", "linear_backward", "distill_forward",
           "distill_backward", "distill_loss_grad", "embedding_forward", "embedding_backward",
           "linear_cross_entropy_forward", "linear_cross_entropy_backward", "linear_cross_entropy_loss_grad", "layer_norm",
           "linear", "distill_loss", "embedding", "linear_cross_entropy", "check", "ACTIVATIONS"]

ACTIVATIONS = {"none": _ops_abi.SOMA_ACT_NONE, "relu": _ops_abi.SOMA_ACT_RELU, "gelu": _ops_abi.SOMA_ACT_GELU,
               "gelu_tanh": _ops_abi.SOMA_ACT_GELU_TANH, "silu": _ops_abi.SOMA_ACT_SILU}

_CODE = {torch.float32: SOMA_DTYPE_F32, torch.bfloat16: SOMA_DTYPE_BF16, torch.float16: SOMA_DTYPE_F16}
_INDEX = {torch.int32: _ops_abi.SOMA_INDEX_I32, torch.int64: _ops_abi.SOMA_INDEX_I64}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check(status: int):
    if status != 0:
        raise SomaError(status, _ops_abi.soma_ops_last_error().decode())


def check(device: int = 0):
    """Waits for the device and raises SomaError if a kernel of these operators
    gave up waiting for its own copies since the last check (its results are
    then not valid; a fault of the library)."""
    _ops_abi.load()
    _check(_ops_abi.soma_ops_check(device))


def _on_stream(fn):
    """Gives an operator its `stream` argument: the call runs with that stream current."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = kwargs.pop("stream", None) if kwargs else None
        if stream is None:
            return fn(*args, **kwargs)
        tensors = [t for t in (*args, *kwargs.values()) if isinstance(t, torch.Tensor)]
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=tensors[0].device)
        with torch.cuda.stream(stream):
            out = fn(*args, **kwargs)
        for t in tensors:  # their memory may not be reused before the call's work is done
            if t.is_cuda:
                t.record_stream(stream)
        return out
    return call


def _code(t, name, among=_CODE) -> int:
    code = among.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} ({', '.join(str(d) for d in among)})")
    return code


def _matrix(t, name):
    """t as [rows, last], without a copy."""
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name}: expected at least one dimension")
        if t.dim() == 1:
            t = t.unsqueeze(0)
        else:
            last, rows = t.shape[-1], 1
            for s in t.shape[:-1]:
                rows *= s
            try:
                t = t.view(rows, last)
            except RuntimeError:
                raise ValueError(f"{name}: its leading dimensions are not evenly spaced rows") from None
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.stride(1) != 1 and t.shape[1] > 1 and t.shape[0] > 0:
        raise ValueError(f"{name}: the last dimension must have unit stride")
    return t


def _like(t, name, other, shape, dtype=None):
    """Checks a tensor that has to match `other`'s device, and its shape and dtype."""
    if t.shape == shape and (dtype is None or t.dtype is dtype) and t.get_device() == other.get_device():
        return
    if t.device != other.device:
        raise ValueError(f"{name}: on {t.device}, expected {other.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")


def _vector(t, name, other, n, dtype):
    """Address of an optional contiguous vector."""
    if t is None:
        return None
    _like(t, name, other, (n,), dtype)
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _empty_rows(like, shape):
    """An output of `shape` for the matrix `like`.  Its rows start at the same
    offsets from a 16-byte boundary as those of `like`, so that the kernel can
    move whole vectors of both: contiguous when `like` is, else padded by less
    than 16 bytes a row."""
    rows, cols = like.shape
    per = 16 // like.element_size()
    stride = like.stride(0)
    if stride == cols or rows <= 1 or (stride - cols) % per == 0:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    stride = cols + (stride - cols) % per
    out = torch.empty((rows, stride), dtype=like.dtype, device=like.device)[:, :cols]
    return out if len(shape) == 2 else out.unflatten(0, shape[:-1])


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


# Workspace sizes depend on sizes and alignment alone: asked once per combination.

def _unaligned(t) -> bool:
    """Whether a 16-bit matrix has rows that do not start on 16-byte boundaries."""
    return t.data_ptr() % 16 != 0 or (t.stride(0) % 8 != 0 and t.shape[0] > 1)


def _operand(unaligned: bool, cols: int):
    """(address, stride) of some matrix with aligned or unaligned rows, to ask for sizes with."""
    return (2, cols) if unaligned else (16, (cols + 7) // 8 * 8)


@functools.lru_cache(maxsize=1024)
def _norm_bytes(dev, rows, cols):
    need = ctypes.c_int64()
    _check(_ops_abi.soma_layer_norm_backward_workspace(dev, rows, cols, ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=1024)
def _linear_forward_bytes(dev, m, n, k, dt, x, w):
    need = ctypes.c_int64()
    _check(_ops_abi.soma_linear_forward_workspace(dev, *_operand(x, k), *_operand(w, k), m, n, k, dt,
                                                  ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=1024)
def _linear_backward_bytes(dev, m, n, k, dt, act, dy, x, w):
    need = ctypes.c_int64()
    _check(_ops_abi.soma_linear_backward_workspace(dev, *_operand(dy, n), *_operand(x, k), *_operand(w, k), m, n, k,
                                                   dt, act, ctypes.byref(need)))
    return need.value


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---- layer norm -------------------------------------------------------------

@_on_stream
def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5):
    """(y, mean, rstd) of a layer norm over the last dimension.

    x: fp32, bf16 or fp16.  weight, bias: fp32 or x's dtype (both the same),
    or None.  y has x's dtype; mean and rstd are fp32, one per row."""
    _ops_abi.load()
    x2 = _matrix(x, "x")
    rows, cols = x2.shape
    param = weight if weight is not None else bias
    wdt = x.dtype if param is None else param.dtype
    w, b = _vector(weight, "weight", x, cols, wdt), _vector(bias, "bias", x, cols, wdt)
    dt = _code(x, "x")
    pdt = dt if param is None else _code(param, "weight")
    y = _empty_rows(x2, x.shape)
    y2 = y if y.dim() == 2 else _matrix(y, "y")
    mean = torch.empty(rows, dtype=torch.float32, device=x.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    dev = x.device.index
    _check(_ops_abi.soma_layer_norm_forward(dev, x2.data_ptr(), x2.stride(0), w, b, y2.data_ptr(), y2.stride(0),
                                            mean.data_ptr(), rstd.data_ptr(), rows, cols, dt, pdt, eps,
                                            _raw_stream(dev)))
    return y, mean, rstd


@_on_stream
def layer_norm_backward(dy, x, weight, mean, rstd, *, input_grad: bool = True, weight_grad: bool = True,
                        bias_grad: bool = True):
    """(dx, dweight, dbias) of layer_norm_forward; mean and rstd are its
    results.  dweight and dbias have the weight's dtype and are None without a
    weight; so is any gradient not asked for."""
    _ops_abi.load()
    x2 = _matrix(x, "x")
    rows, cols = x2.shape
    _like(dy, "dy", x, x.shape, x.dtype)
    dy2 = _matrix(dy, "dy")
    dt = _code(x, "x")
    w = _vector(weight, "weight", x, cols, None)
    pdt = dt if weight is None else _code(weight, "weight")
    m, r = _vector(mean, "mean", x, rows, torch.float32), _vector(rstd, "rstd", x, rows, torch.float32)
    dev = x.device.index
    dx = dx2 = dweight = dbias = work = None
    if input_grad:
        dx = _empty_rows(x2, x.shape)
        dx2 = dx if dx.dim() == 2 else _matrix(dx, "dx")
    if weight is not None and (weight_grad or bias_grad):
        dweight = torch.empty_like(weight) if weight_grad else None
        dbias = torch.empty_like(weight) if bias_grad else None
        work = _workspace(_norm_bytes(dev, rows, cols), x.device)
    _check(_ops_abi.soma_layer_norm_backward(dev, dy2.data_ptr(), dy2.stride(0), x2.data_ptr(), x2.stride(0), w, m, r,
                                             _ptr(dx2), dx2.stride(0) if dx2 is not None else 0, _ptr(dweight),
                                             _ptr(dbias), _ptr(work), work.numel() if work is not None else 0, rows,
                                             cols, dt, pdt, _raw_stream(dev)))
    return dx, dweight, dbias


# ---- linear layer -------------------------------------------------------------

def _activation(name) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return code


@_on_stream
def linear_forward(x, weight, bias=None, *, activation: str = "none", residual=None,
                   save_preactivation: bool = False):
    """y = act(x weight^T + bias) + residual, and with save_preactivation
    (y, z), z = x weight^T + bias for linear_backward.

    x [..., k], weight [n, k], bias [n], residual [..., n]: all bf16 or all
    fp16.  y and z are contiguous."""
    _ops_abi.load()
    x2, w2 = _matrix(x, "x"), _matrix(weight, "weight")
    m, k = x2.shape
    n = w2.shape[0]
    _like(weight, "weight", x, (n, k), x.dtype)
    dt, act = _code(x, "x"), _activation(activation)
    b = _vector(bias, "bias", x, n, x.dtype)
    shape = (*x.shape[:-1], n)
    r2 = None
    if residual is not None:
        _like(residual, "residual", x, shape, x.dtype)
        r2 = _matrix(residual, "residual")
    y = torch.empty(shape, dtype=x.dtype, device=x.device)
    z = torch.empty_like(y) if save_preactivation else None
    dev = x.device.index
    need = _linear_forward_bytes(dev, m, n, k, dt, _unaligned(x2), _unaligned(w2))
    work = _workspace(need, x.device)
    _check(_ops_abi.soma_linear_forward(dev, x2.data_ptr(), x2.stride(0), w2.data_ptr(), w2.stride(0), b, _ptr(r2),
                                        r2.stride(0) if r2 is not None else 0, y.data_ptr(), n, _ptr(z), n,
                                        _ptr(work), need, m, n, k, dt, act, _raw_stream(dev)))
    return (y, z) if save_preactivation else y


@_on_stream
def linear_backward(dy, x, weight, preactivation=None, *, activation: str = "none", input_grad: bool = True,
                    weight_grad: bool = True, bias_grad: bool = True):
    """(dx, dweight, dbias) of linear_forward (the residual's gradient is dy).

    preactivation: z of the forward pass, needed with an activation.  The
    gradients have x's dtype; those not asked for are None."""
    _ops_abi.load()
    x2, w2 = _matrix(x, "x"), _matrix(weight, "weight")
    m, k = x2.shape
    n = w2.shape[0]
    _like(weight, "weight", x, (n, k), x.dtype)
    shape = (*x.shape[:-1], n)
    _like(dy, "dy", x, shape, x.dtype)
    dy2 = _matrix(dy, "dy")
    dt, act = _code(x, "x"), _activation(activation)
    z2 = None
    if act != _ops_abi.SOMA_ACT_NONE:
        if preactivation is None:
            raise ValueError(f"preactivation: needed for the gradient of {activation}")
        _like(preactivation, "preactivation", x, shape, x.dtype)
        z2 = _matrix(preactivation, "preactivation")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if input_grad else None
    dw = torch.empty((n, k), dtype=x.dtype, device=x.device) if weight_grad else None
    db = torch.empty(n, dtype=x.dtype, device=x.device) if bias_grad else None
    dev = x.device.index
    need = _linear_backward_bytes(dev, m, n, k, dt, act, _unaligned(dy2), _unaligned(x2), _unaligned(w2))
    work = _workspace(need, x.device)
    _check(_ops_abi.soma_linear_backward(dev, dy2.data_ptr(), dy2.stride(0), x2.data_ptr(), x2.stride(0),
                                         w2.data_ptr(), w2.stride(0), _ptr(z2), z2.stride(0) if z2 is not None else 0,
                                         _ptr(dx), k, _ptr(dw), k, _ptr(db), _ptr(work), need, m, n, k, dt, act,
                                         _raw_stream(dev)))
    return dx, dw, db


# ---- distillation loss ----------------------------------------------------------

def _distill_inputs(logits, teacher_logits, teacher_index, row_weight):
    """The arguments that the three calls share: (rows view, what the C calls take before and after the outputs)."""
    z = _matrix(logits, "logits")
    rows, vocab = z.shape
    t, i = _matrix(teacher_logits, "teacher_logits"), _matrix(teacher_index, "teacher_index")
    top = t.shape[1]
    _like(teacher_logits, "teacher_logits", logits, (*logits.shape[:-1], top))
    _like(teacher_index, "teacher_index", logits, (*logits.shape[:-1], top))
    w = None
    if row_weight is not None:
        _like(row_weight, "row_weight", logits, logits.shape[:-1], torch.float32)
        if not row_weight.is_contiguous():
            raise ValueError("row_weight: must be contiguous")
        w = row_weight.data_ptr()
    first = (z.data_ptr(), z.stride(0))
    middle = (t.data_ptr(), t.stride(0), i.data_ptr(), i.stride(0), w)
    last = (rows, vocab, top, _code(logits, "logits"), _code(teacher_logits, "teacher_logits"),
            _code(teacher_index, "teacher_index", _INDEX))
    return z, first, middle, last


def _out_rows(z, logits, out):
    """(output, its address and stride) for dlogits: a new tensor, or `out`."""
    if out is None:
        out = _empty_rows(z, logits.shape)
    else:
        _like(out, "out", logits, logits.shape, logits.dtype)
    o2 = out if out.dim() == 2 else _matrix(out, "out")
    return out, o2.data_ptr(), o2.stride(0)


def _written(out):
    """Tells autograd that a tensor of the caller's has changed: a graph that saved it refuses its backward pass."""
    if out is not None and not out.is_inference():
        torch.autograd.graph.increment_version(out)


@_on_stream
def distill_forward(logits, teacher_logits, teacher_index, *, temperature: float = 1.0, row_weight=None):
    """(loss, lse), fp32 and one per row: the temperature-scaled divergence of
    the student's distribution over the vocabulary from the teacher's over its
    top entries, and the log of the student's normalizer.

    logits [..., vocab]; teacher_logits and teacher_index (int32 or int64)
    [..., top]; an index outside the vocabulary, such as -1, marks an entry
    that does not count.  row_weight [...] fp32: a row of weight 0 is not read
    and gets loss, lse and gradient 0."""
    _ops_abi.load()
    _, first, middle, last = _distill_inputs(logits, teacher_logits, teacher_index, row_weight)
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    lse = torch.empty_like(loss)
    dev = logits.device.index
    _check(_ops_abi.soma_distill_forward(dev, *first, *middle, temperature, loss.data_ptr(), lse.data_ptr(), *last,
                                         _raw_stream(dev)))
    return loss, lse


@_on_stream
def distill_backward(grad_loss, logits, lse, teacher_logits, teacher_index, *, temperature: float = 1.0,
                     row_weight=None, out=None):
    """dL/dlogits for grad_loss = dL/dloss; lse is distill_forward's.  out may
    be `logits`: the gradient then takes the logits' place (autograd counts
    that as a change in place)."""
    _ops_abi.load()
    z, first, middle, last = _distill_inputs(logits, teacher_logits, teacher_index, row_weight)
    for t, name in ((grad_loss, "grad_loss"), (lse, "lse")):
        _like(t, name, logits, logits.shape[:-1], torch.float32)
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    gradient, address, stride = _out_rows(z, logits, out)
    dev = logits.device.index
    _check(_ops_abi.soma_distill_backward(dev, grad_loss.data_ptr(), *first, lse.data_ptr(), *middle, temperature,
                                          address, stride, *last, _raw_stream(dev)))
    _written(out)
    return gradient


@_on_stream
def distill_loss_grad(logits, teacher_logits, teacher_index, *, temperature: float = 1.0, row_weight=None, out=None):
    """(loss, dlogits) in one kernel: distill_forward's loss and the gradient
    of its sum (put 1 / (number of rows), a loss scale and the like into
    row_weight).  out may be `logits`."""
    _ops_abi.load()
    z, first, middle, last = _distill_inputs(logits, teacher_logits, teacher_index, row_weight)
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    gradient, address, stride = _out_rows(z, logits, out)
    dev = logits.device.index
    _check(_ops_abi.soma_distill_loss_grad(dev, *first, *middle, temperature, loss.data_ptr(), None, address, stride,
                                           *last, _raw_stream(dev)))
    _written(out)
    return loss, gradient


# ---- embedding ----------------------------------------------------------------

def _tokens(t, name, other):
    """Token numbers of any shape as the C calls take them: (address, stride, batch, length, type)."""
    code = _code(t, name, _INDEX)
    if t.device != other.device:
        raise ValueError(f"{name}: on {t.device}, expected {other.device}")
    if t.dim() == 1 and t.is_cuda and t.is_contiguous():  # (host time: most calls)
        n = t.shape[0]
        return t.data_ptr(), n, 1, n, code
    if t.dim() == 1 and t.is_cuda and t.stride(0) > 0:  # one token of each text
        return t.data_ptr(), t.stride(0), t.shape[0], 1, code
    if t.dim() == 0:
        t = t.unsqueeze(0)
    m = _matrix(t, name)
    return m.data_ptr(), m.stride(0), m.shape[0], m.shape[1], code


@functools.lru_cache(maxsize=1024)
def _embedding_bytes(dev, rows, vocab, cols):
    need = ctypes.c_int64()
    _check(_ops_abi.soma_embedding_backward_workspace(dev, rows, vocab, cols, ctypes.byref(need)))
    return need.value


@_on_stream
def embedding_forward(index, weight, *, scale: float = 1.0):
    """y = scale * weight[index], [..., cols] in the weight's dtype.

    index [...]: int32 or int64; a token outside the vocabulary, such as -1,
    gets zeros.  weight [vocab, cols]: fp32, bf16 or fp16."""
    _ops_abi.load()
    if weight.dim() != 2:
        raise ValueError(f"weight: {weight.dim()} dimensions, expected 2")
    w = _matrix(weight, "weight")
    vocab, cols = w.shape
    address, stride, batch, length, code = _tokens(index, "index", weight)
    y = torch.empty((*index.shape, cols), dtype=weight.dtype, device=weight.device)
    dev = weight.device.index
    _check(_ops_abi.soma_embedding_forward(dev, w.data_ptr(), w.stride(0), address, stride, batch, length, y.data_ptr(),
                                           cols, vocab, cols, _code(weight, "weight"), code, scale, _raw_stream(dev)))
    return y


@_on_stream
def embedding_backward(dy, index, vocab: int, *, scale: float = 1.0, out=None):
    """dweight [vocab, cols] of embedding_forward, in dy's dtype; summed in
    fp32.  With `out` (such as the gradient of a last linear layer that shares
    the table) the gradient is added to it, and it is returned."""
    _ops_abi.load()
    d = _matrix(dy, "dy")
    cols = d.shape[1]
    _like(dy, "dy", dy, (*index.shape, cols))
    address, stride, batch, length, code = _tokens(index, "index", dy)
    dt = _code(dy, "dy")
    dweight = out
    if out is None:
        dweight = torch.empty((vocab, cols), dtype=dy.dtype, device=dy.device)
    else:
        _like(out, "out", dy, (vocab, cols), dy.dtype)
    w = _matrix(dweight, "out")
    dev = dy.device.index
    need = _embedding_bytes(dev, batch * length, vocab, cols)
    work = _workspace(need, dy.device)
    _check(_ops_abi.soma_embedding_backward(dev, d.data_ptr(), d.stride(0), address, stride, batch, length, w.data_ptr(),
                                            w.stride(0), int(out is not None), _ptr(work), need, vocab, cols, dt, code,
                                            scale, _raw_stream(dev)))
    _written(out)
    return dweight


# ---- cross entropy of a linear layer ---------------------------------------------

@functools.lru_cache(maxsize=1024)
def _head_bytes(dev, w, rows, vocab, k, dt, forward, dx, dweight):
    need = ctypes.c_int64()
    _check(_ops_abi.soma_linear_cross_entropy_workspace(dev, *_operand(w, k), rows, vocab, k, dt, forward, dx, dweight,
                                                        ctypes.byref(need)))
    return need.value


def _head_inputs(x, weight, target, row_weight, forward, dx, dweight):
    """What the three calls share: (device, what the C calls take first, row weights, workspace, what they take last)."""
    x2 = _matrix(x, "x")
    w2 = _matrix(weight, "weight")
    rows, k = x2.shape
    vocab = w2.shape[0]
    _like(weight, "weight", x, (vocab, k), x.dtype)
    if target.shape != x.shape[:-1]:
        raise ValueError(f"target: shape {tuple(target.shape)}, expected {tuple(x.shape[:-1])}")
    address, stride, batch, length, code = _tokens(target, "target", x)
    w = None
    if row_weight is not None:
        _like(row_weight, "row_weight", x, x.shape[:-1], torch.float32)
        if not row_weight.is_contiguous():
            raise ValueError("row_weight: must be contiguous")
        w = row_weight.data_ptr()
    dt = _code(x, "x")
    dev = x.device.index
    need = _head_bytes(dev, _unaligned(w2), rows, vocab, k, dt, int(forward), int(dx), int(dweight))
    first = (x2.data_ptr(), x2.stride(0), w2.data_ptr(), w2.stride(0), address, stride, batch, length)
    return dev, first, w, _workspace(need, x.device), need, (vocab, k, dt, code)


def _head_gradients(x, weight, dx, dweight):
    """New gradients, and (address, stride) of both."""
    k = x.shape[-1]
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if dx else None
    dw = torch.empty(weight.shape, dtype=x.dtype, device=x.device) if dweight else None
    return dx, dw, (_ptr(dx), k, _ptr(dw), k)


@_on_stream
def linear_cross_entropy_forward(x, weight, target, *, row_weight=None):
    """(loss, lse), fp32 and one per row: the cross entropy of softmax(x
    weight^T) at the target tokens, without the logits in memory.

    x [..., k] and weight [vocab, k]: bf16 or fp16.  target [...]: int32 or
    int64; a target outside the vocabulary, such as -100, or a row_weight (fp32,
    [...]) of 0 marks a row that does not count: loss, lse and gradient are 0."""
    _ops_abi.load()
    dev, first, w, work, need, last = _head_inputs(x, weight, target, row_weight, True, False, False)
    loss = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    _check(_ops_abi.soma_linear_cross_entropy_forward(dev, *first, w, loss.data_ptr(), lse.data_ptr(), _ptr(work), need,
                                                      *last, _raw_stream(dev)))
    return loss, lse


@_on_stream
def linear_cross_entropy_backward(grad_loss, x, weight, target, lse, *, row_weight=None, input_grad: bool = True,
                                  weight_grad: bool = True):
    """(dx, dweight) for grad_loss = dL/dloss, in x's dtype; lse is the
    forward pass's.  Those not asked for are None."""
    _ops_abi.load()
    dev, first, w, work, need, last = _head_inputs(x, weight, target, row_weight, False, input_grad, weight_grad)
    for t, name in ((grad_loss, "grad_loss"), (lse, "lse")):
        _like(t, name, x, x.shape[:-1], torch.float32)
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    dx, dw, out = _head_gradients(x, weight, input_grad, weight_grad)
    _check(_ops_abi.soma_linear_cross_entropy_backward(dev, grad_loss.data_ptr(), *first, lse.data_ptr(), w, *out,
                                                       _ptr(work), need, *last, _raw_stream(dev)))
    return dx, dw


@_on_stream
def linear_cross_entropy_loss_grad(x, weight, target, *, row_weight=None, input_grad: bool = True,
                                   weight_grad: bool = True):
    """(loss, dx, dweight): the forward pass and the gradients of the losses'
    sum (put 1 / (number of rows), a loss scale and the like into row_weight)."""
    _ops_abi.load()
    dev, first, w, work, need, last = _head_inputs(x, weight, target, row_weight, True, input_grad, weight_grad)
    loss = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    dx, dw, out = _head_gradients(x, weight, input_grad, weight_grad)
    _check(_ops_abi.soma_linear_cross_entropy_loss_grad(dev, *first, w, loss.data_ptr(), None, *out, _ptr(work), need,
                                                        *last, _raw_stream(dev)))
    return loss, dx, dw


# ---- autograd -----------------------------------------------------------------

def _even(g):
    """An incoming gradient as evenly spaced rows (autograd may hand over expanded or permuted ones)."""
    try:
        if _matrix(g, "gradient").stride(0) >= g.shape[-1]:
            return g
    except ValueError:
        pass
    return g.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        wants = ctx.needs_input_grad
        if weight is None and wants[2]:  # a bias alone: its gradient has the bias's type
            weight = torch.ones(x.shape[-1], dtype=ctx.bias_dtype, device=x.device)
        dx, dw, db = layer_norm_backward(_even(dy), x, weight, mean, rstd, input_grad=wants[0], weight_grad=wants[1],
                                         bias_grad=wants[2])
        return dx, dw, db, None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, residual):
        z = None
        # (the residual's gradient needs no pre-activation)
        if activation != "none" and any(ctx.needs_input_grad[:3]):
            y, z = linear_forward(x, weight, bias, activation=activation, residual=residual, save_preactivation=True)
        else:
            y = linear_forward(x, weight, bias, activation=activation, residual=residual)
        ctx.save_for_backward(x, weight, z)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, z = ctx.saved_tensors
        wants = ctx.needs_input_grad
        dx = dw = db = None
        if any(wants[:3]):
            dx, dw, db = linear_backward(_even(dy), x, weight, z, activation=ctx.activation, input_grad=wants[0],
                                         weight_grad=wants[1], bias_grad=wants[2])
        return dx, dw, db, None, dy if wants[4] else None


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_logits, teacher_index, temperature, row_weight):
        loss, lse = distill_forward(logits, teacher_logits, teacher_index, temperature=temperature,
                                    row_weight=row_weight)
        ctx.save_for_backward(logits, lse, teacher_logits, teacher_index, row_weight)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss):
        logits, lse, teacher_logits, teacher_index, row_weight = ctx.saved_tensors
        return distill_backward(grad_loss.contiguous(), logits, lse, teacher_logits, teacher_index,
                                temperature=ctx.temperature, row_weight=row_weight), None, None, None, None


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, index, weight, scale):
        ctx.save_for_backward(index)
        ctx.vocab, ctx.scale = weight.shape[0], scale
        return embedding_forward(index, weight, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        index, = ctx.saved_tensors
        return None, embedding_backward(_even(dy), index, ctx.vocab, scale=ctx.scale), None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, target, row_weight):
        loss, lse = linear_cross_entropy_forward(x, weight, target, row_weight=row_weight)
        ctx.save_for_backward(x, weight, target, lse, row_weight)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss):
        x, weight, target, lse, row_weight = ctx.saved_tensors
        wants = ctx.needs_input_grad
        dx, dw = linear_cross_entropy_backward(grad_loss.contiguous(), x, weight, target, lse, row_weight=row_weight,
                                               input_grad=wants[0], weight_grad=wants[1])
        return dx, dw, None, None


def layer_norm(x, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, eps: float = 1e-5):
    """Differentiable layer norm over the last dimension (see layer_norm_forward)."""
    return _LayerNorm.apply(x, weight, bias, eps)


def linear(x, weight, bias: Optional[torch.Tensor] = None, *, activation: str = "none",
           residual: Optional[torch.Tensor] = None):
    """Differentiable act(x weight^T + bias) + residual (see linear_forward)."""
    if not torch.is_grad_enabled():  # (needs_input_grad does not know)
        return linear_forward(x, weight, bias, activation=activation, residual=residual)
    return _Linear.apply(x, weight, bias, activation, residual)


def distill_loss(logits, teacher_logits, teacher_index, *, temperature: float = 1.0,
                 row_weight: Optional[torch.Tensor] = None):
    """Differentiable distillation loss per row (see distill_forward); the
    teacher and the row weights are constants."""
    return _Distill.apply(logits, teacher_logits, teacher_index, temperature, row_weight)


def embedding(index, weight, *, scale: float = 1.0):
    """Differentiable scale * weight[index] (see embedding_forward)."""
    return _Embedding.apply(index, weight, scale)


def linear_cross_entropy(x, weight, target, *, row_weight: Optional[torch.Tensor] = None):
    """Differentiable cross entropy per row of softmax(x weight^T) (see
    linear_cross_entropy_forward); the row weights are constants."""
    return _LinearCrossEntropy.apply(x, weight, target, row_weight)
