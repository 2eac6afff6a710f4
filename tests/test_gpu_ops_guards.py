"""The training operators write their outputs and nothing else: through the C ABI, every output and workspace lies inside a
larger buffer (rows with gaps, odd starts) whose other bytes must not change, and the values are those of the Python calls."""
import ctypes
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu
CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
PLACES = [(0, 0), (1, 0), (3, 1), (8, 0), (8, 3), (40, 8)]  # gap between rows, first element's offset
GUARD = 64                                                  # elements before and after


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


@pytest.fixture(scope="module")
def C(ops):
    from tensor_grad_clip_gb300 import _ops_abi
    _ops_abi.load()
    return _ops_abi


class Output:
    """[rows, cols] in a buffer of a pattern; changed() is what was written outside of it."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0):
        self.stride, size = cols + pad, dtype.itemsize
        n = GUARD + offset + rows * self.stride + GUARD
        bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[size]
        pattern = torch.arange(n, device="cuda") * 40503 % 30011 + 100
        self.raw = pattern.to(bits) if size > 1 else (pattern % 251).to(bits)
        self.before = self.raw.clone()
        self.span = slice(GUARD + offset, GUARD + offset + rows * self.stride)
        self.rows, self.cols, self.dtype = rows, cols, dtype
        self.at = self.raw.data_ptr() + (GUARD + offset) * size

    def value(self):
        return self.raw[self.span].view(self.rows, self.stride)[:, :self.cols].contiguous().view(self.dtype)

    def changed(self):
        mine = torch.zeros_like(self.raw, dtype=torch.bool)
        mine[self.span].view(self.rows, self.stride)[:, :self.cols] = True
        return int(((self.raw != self.before) & ~mine).sum())


def same(output, want, what):
    assert output.changed() == 0, f"{what}: {output.changed()} elements written outside"
    bits = torch.int32 if output.dtype == torch.float32 else torch.int16
    got = output.value().view(want.shape)
    assert torch.equal(got.view(bits), want.contiguous().view(bits)), what


def inputs(rows, cols, dtype, pad, offset, std=1.0):
    buf = torch.randn(rows * (cols + pad) + offset, device="cuda").mul(std).to(dtype)
    return buf[offset:].view(rows, cols + pad)[:, :cols]


def ptr(t):
    return None if t is None else t.at if isinstance(t, Output) else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def workspace(nbytes):
    """A guarded workspace; it starts on a 256-byte boundary."""
    w = Output(1, max(1, nbytes), torch.uint8, 0, 192)
    assert w.at % 256 == 0
    return w


@pytest.mark.parametrize("pad,offset", PLACES)
@pytest.mark.parametrize("dtype", list(CODE))
def test_layer_norm(ops, C, dtype, pad, offset):
    for rows, cols in itertools.product((1, 5, 700), (1, 31, 96, 500, 1000, 1024, 4099, 8200, 16384, 16391)):
        if rows == 700 and cols > 4099:
            continue
        x, dy = inputs(rows, cols, dtype, pad, offset), inputs(rows, cols, dtype, pad, offset)
        w, b = torch.rand(cols, device="cuda"), torch.rand(cols, device="cuda")
        want = ops.layer_norm_forward(x, w, b)
        y, mean, rstd = Output(rows, cols, dtype, pad, offset), *(Output(1, rows, torch.float32, 0, offset) for _ in "mr")
        assert C.soma_layer_norm_forward(0, ptr(x), cols + pad, ptr(w), ptr(b), ptr(y), y.stride, ptr(mean), ptr(rstd),
                                         rows, cols, CODE[dtype], 0, 1e-5, stream()) == 0
        for o, v, name in zip((y, mean, rstd), want, ("y", "mean", "rstd")):
            same(o, v, f"{name} {rows}x{cols}")
        want = ops.layer_norm_backward(dy, x, w, want[1], want[2])
        mu, rs = mean.value().view(-1), rstd.value().view(-1)
        need = ctypes.c_int64()
        assert C.soma_layer_norm_backward_workspace(0, rows, cols, ctypes.byref(need)) == 0
        ws = workspace(need.value)
        dx, dw, db = Output(rows, cols, dtype, pad, offset), *(Output(1, cols, torch.float32, 0, offset) for _ in "wb")
        assert C.soma_layer_norm_backward(0, ptr(dy), cols + pad, ptr(x), cols + pad, ptr(w), ptr(mu), ptr(rs), ptr(dx),
                                          dx.stride, ptr(dw), ptr(db), ptr(ws), need.value, rows, cols, CODE[dtype], 0,
                                          stream()) == 0
        for o, v, name in zip((dx, dw, db), want, ("dx", "dweight", "dbias")):
            same(o, v, f"{name} {rows}x{cols}")
        assert ws.changed() == 0, "outside the workspace"


@pytest.mark.parametrize("pad,offset", PLACES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear(ops, C, dtype, pad, offset):
    # one row to many tiles, by both kernels; widths that end inside a tile, a box and a 16-byte word
    for m, n, k in ((1, 8, 8), (1, 1000, 72), (17, 131, 100), (64, 264, 520), (130, 257, 65), (300, 1016, 264),
                    (513, 769, 129), (700, 2056, 136), (2100, 2300, 72)):
        x, w = inputs(m, k, dtype, pad, offset), inputs(n, k, dtype, pad, offset, k ** -0.5)
        r, dy, b = inputs(m, n, dtype, pad, offset), inputs(m, n, dtype, pad, offset), torch.randn(n, device="cuda").to(dtype)
        want = ops.linear_forward(x, w, b, activation="silu", residual=r, save_preactivation=True)
        need = ctypes.c_int64()
        assert C.soma_linear_forward_workspace(0, ptr(x), k + pad, ptr(w), k + pad, m, n, k, CODE[dtype],
                                               ctypes.byref(need)) == 0
        ws = workspace(need.value)
        y, z = Output(m, n, dtype, pad, offset), Output(m, n, dtype, pad, offset)
        assert C.soma_linear_forward(0, ptr(x), k + pad, ptr(w), k + pad, ptr(b), ptr(r), n + pad, ptr(y), y.stride, ptr(z),
                                     z.stride, ptr(ws), need.value, m, n, k, CODE[dtype], C.SOMA_ACT_SILU, stream()) == 0
        same(y, want[0], f"y {m}x{n}x{k}")
        same(z, want[1], f"z {m}x{n}x{k}")
        assert ws.changed() == 0, "outside the workspace"
        want = ops.linear_backward(dy, x, w, r, activation="silu")
        assert C.soma_linear_backward_workspace(0, ptr(dy), n + pad, ptr(x), k + pad, ptr(w), k + pad, m, n, k, CODE[dtype],
                                                C.SOMA_ACT_SILU, ctypes.byref(need)) == 0
        ws = workspace(need.value)
        dx, dw = Output(m, k, dtype, pad, offset), Output(n, k, dtype, pad, offset)
        db = Output(1, n, dtype, 0, offset)
        assert C.soma_linear_backward(0, ptr(dy), n + pad, ptr(x), k + pad, ptr(w), k + pad, ptr(r), n + pad, ptr(dx),
                                      dx.stride, ptr(dw), dw.stride, ptr(db), ptr(ws), need.value, m, n, k, CODE[dtype],
                                      C.SOMA_ACT_SILU, stream()) == 0
        for o, v, name in zip((dx, dw, db), want, ("dx", "dweight", "dbias")):
            same(o, v, f"{name} {m}x{n}x{k}")
        assert ws.changed() == 0, "outside the workspace"


@pytest.mark.parametrize("pad,offset", PLACES)
def test_linear_gradients_of_nothing(C, pad, offset):
    for m, n in ((0, 24), (5, 0)):
        k = 40
        dx, dw = Output(max(m, 1), k, torch.float16, pad, offset), Output(max(n, 1), k, torch.float16, pad, offset)
        db = Output(1, max(n, 1), torch.float16, 0, offset)
        x, w = (inputs(rows, k, torch.float16, pad, offset) if rows else None for rows in (m, n))  # (NULL where it has no rows)
        assert C.soma_linear_backward(0, None, n + pad, ptr(x), k + pad, ptr(w), k + pad, None, 0, ptr(dx), dx.stride,
                                      ptr(dw), dw.stride, ptr(db), None, 0, m, n, k, 2, C.SOMA_ACT_NONE, stream()) == 0
        for o, written in ((dx, m > 0), (dw, n > 0), (db, n > 0)):
            assert o.changed() == 0
            assert not o.value().any() if written else torch.equal(o.raw, o.before)


@pytest.mark.parametrize("pad,offset", PLACES)
@pytest.mark.parametrize("dtype", list(CODE))
def test_distillation(ops, C, dtype, pad, offset):
    # few rows (a cluster each), rows of a CTA, and enough long rows for the persistent kernel
    shapes = [(1, 1), (3, 7), (2, 40000), (5, 4099), (40, 1000), (700, 300)]
    shapes += [(620, 16400 if dtype != torch.float32 else 8200), (620, 50003)] if (pad, offset) in PLACES[2:4] else []
    for rows, vocab in shapes:
        top = min(vocab, 12)
        z = inputs(rows, vocab, dtype, pad, offset, 2.5)
        t, index = torch.randn(rows, top, device="cuda"), torch.randint(-1, vocab, (rows, top), device="cuda").int()
        w, g = torch.rand(rows, device="cuda"), torch.randn(rows, device="cuda")
        w[rows // 2] = 0 if rows > 1 else 1
        loss, lse = ops.distill_forward(z, t, index, temperature=1.5, row_weight=w)
        both = ops.distill_loss_grad(z, t, index, temperature=1.5, row_weight=w)
        grad = ops.distill_backward(g, z, lse, t, index, temperature=1.5, row_weight=w)
        head = (ptr(z), vocab + pad)
        teacher = (ptr(t), top, ptr(index), top, ptr(w), 1.5)
        tail = (rows, vocab, top, CODE[dtype], 0, 0, stream())
        l1, e1, l2, e2 = (Output(1, rows, torch.float32, 0, offset) for _ in range(4))
        d1, d2 = (Output(rows, vocab, dtype, pad, offset) for _ in range(2))
        assert C.soma_distill_forward(0, *head, *teacher, ptr(l1), ptr(e1), *tail) == 0
        assert C.soma_distill_loss_grad(0, *head, *teacher, ptr(l2), ptr(e2), ptr(d1), d1.stride, *tail) == 0
        assert C.soma_distill_backward(0, ptr(g), *head, ptr(lse), *teacher, ptr(d2), d2.stride, *tail) == 0
        for o, v, name in ((l1, loss, "loss"), (e1, lse, "lse"), (l2, both[0], "loss of both"), (d1, both[1], "gradient of both"),
                           (d2, grad, "gradient")):
            same(o, v, f"{name} {rows}x{vocab}")
        assert e2.changed() == 0
