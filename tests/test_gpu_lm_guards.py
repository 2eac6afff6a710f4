"""The embedding and the linear layer with cross entropy write their outputs and nothing else, also past 32-bit offsets: through
the C ABI, every output and workspace lies inside a larger buffer whose other bytes must not change."""
import ctypes

import pytest
import torch

from test_gpu_ops_guards import CODE, PLACES, Output, inputs, ptr, same, stream, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


@pytest.fixture(scope="module")
def C(ops):
    from tensor_grad_clip_gb300 import _ops_abi
    _ops_abi.load()
    return _ops_abi


def ok(status, C):
    assert status == 0, C.soma_ops_last_error().decode()


@pytest.mark.parametrize("pad,offset", PLACES)
@pytest.mark.parametrize("dtype", list(CODE))
def test_embedding(ops, C, dtype, pad, offset):
    for rows, vocab, cols in ((70, 40, 64), (33, 65, 37), (300, 9, 1), (5000, 100, 24)):
        table, dy = inputs(vocab, cols, dtype, pad, offset), inputs(rows, cols, dtype, pad, offset)
        index = torch.randint(-2, vocab + 2, (rows,), device="cuda")
        y, dw = Output(rows, cols, dtype, pad, offset), Output(vocab, cols, dtype, pad, offset)
        ok(C.soma_embedding_forward(0, ptr(table), cols + pad, ptr(index), rows, 1, rows, ptr(y), cols + pad, vocab, cols,
                                    CODE[dtype], 1, 0.5, stream()), C)
        need = ctypes.c_int64()
        ok(C.soma_embedding_backward_workspace(0, rows, vocab, cols, ctypes.byref(need)), C)
        work = workspace(need.value)
        ok(C.soma_embedding_backward(0, ptr(dy), cols + pad, ptr(index), rows, 1, rows, ptr(dw), cols + pad, 0, ptr(work),
                                     need.value, vocab, cols, CODE[dtype], 1, 0.5, stream()), C)
        same(y, ops.embedding_forward(index, table, scale=0.5), "y")
        same(dw, ops.embedding_backward(dy, index, vocab, scale=0.5), "dweight")
        assert work.changed() == 0


@pytest.mark.parametrize("pad,offset", PLACES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_cross_entropy(ops, C, dtype, pad, offset):
    for rows, vocab, k in ((70, 40, 64), (3, 300, 37), (200, 33, 129), (1024, 2500, 72)):
        x, w = inputs(rows, k, dtype, pad, offset), inputs(vocab, k, dtype, pad, offset, 0.1)
        t = torch.randint(-2, vocab + 2, (rows,), device="cuda", dtype=torch.int32)
        g = torch.randn(rows, device="cuda")
        weight = torch.rand(rows, device="cuda")
        weight[::5] = 0
        loss, lse = Output(1, rows, torch.float32), Output(1, rows, torch.float32)
        dx, dw = Output(rows, k, dtype, pad, offset), Output(vocab, k, dtype, pad, offset)

        def run(forward, name, before, middle, outs):
            need = ctypes.c_int64()
            ok(C.soma_linear_cross_entropy_workspace(0, ptr(w), k + pad, rows, vocab, k, CODE[dtype], forward,
                                                     *((1, 1) if dx in outs else (0, 0)), ctypes.byref(need)), C)
            work = workspace(need.value)
            args = [0, *before, ptr(x), k + pad, ptr(w), k + pad, ptr(t), rows, 1, rows, *middle]
            for o in outs:
                args += [ptr(o), k + pad] if o in (dx, dw) else [ptr(o)]
            ok(getattr(C, "soma_linear_cross_entropy_" + name)(*args, ptr(work), need.value, vocab, k, CODE[dtype], 0,
                                                               stream()), C)
            assert work.changed() == 0, name
        kw = dict(row_weight=weight)
        run(1, "forward", [], [ptr(weight)], [loss, lse])
        want_loss, want_lse = ops.linear_cross_entropy_forward(x, w, t, **kw)
        same(loss, want_loss, "loss")
        same(lse, want_lse, "lse")
        run(0, "backward", [ptr(g)], [ptr(want_lse), ptr(weight)], [dx, dw])
        want = ops.linear_cross_entropy_backward(g, x, w, t, want_lse, **kw)
        same(dx, want[0], "dx")
        same(dw, want[1], "dweight")
        run(1, "loss_grad", [], [ptr(weight)], [loss, lse, dx, dw])
        want = ops.linear_cross_entropy_loss_grad(x, w, t, **kw)
        same(loss, want[0], "loss")
        same(lse, want_lse, "lse")
        same(dx, want[1], "dx")
        same(dw, want[2], "dweight")


def test_a_table_past_2_to_the_31_elements(ops):
    vocab, cols = 530_000, 4096
    table = torch.zeros(vocab, cols, dtype=torch.bfloat16, device="cuda")
    table[-3:] = torch.randn(3, cols, device="cuda").bfloat16()
    index = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 1, vocab], device="cuda")
    y = ops.embedding_forward(index, table)
    assert torch.equal(y[0], table[-1]) and torch.equal(y[2], table[-3]) and not y[[1, 4]].any()
    dy = torch.randn(5, cols, device="cuda").bfloat16()
    d = ops.embedding_backward(dy, index, vocab)
    assert torch.equal(d[-1], (dy[0].float() + dy[3].float()).bfloat16()) and torch.equal(d[-3], dy[2])
    assert torch.equal(d[0], dy[1]) and not d[1:-3].any() and not d[-2].any()


def test_rows_and_weights_past_2_to_the_31_elements(ops):
    torch.manual_seed(1)
    # rows of x and of the weight far apart, and a weight's gradient of more than 2^31 elements
    rows, vocab, k, gap = 300, 700, 64, 7_200_000
    buf = torch.empty(rows * gap, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, gap)[:, :k]
    x.copy_(torch.randn(rows, k, device="cuda"))
    w, t = torch.randn(vocab, k, device="cuda").bfloat16(), torch.randint(0, vocab, (rows,), device="cuda")
    a, b = (ops.linear_cross_entropy_loss_grad(v, w, t) for v in (x, x.contiguous()))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    wide = torch.empty(vocab * 3_200_000, dtype=torch.bfloat16, device="cuda").view(vocab, 3_200_000)[:, :k]
    wide.copy_(w)
    c = ops.linear_cross_entropy_loss_grad(x, wide, t)
    assert all(torch.equal(p, q) for p, q in zip(b, c))
    del buf, x, wide
    vocab, k = 530_000, 4096
    w = torch.zeros(vocab, k, dtype=torch.bfloat16, device="cuda")
    w[-5:] = torch.randn(5, k, device="cuda").bfloat16() / 16
    x = torch.randn(4, k, device="cuda").bfloat16()
    t = torch.tensor([vocab - 1, vocab - 5, 0, vocab - 2], device="cuda")
    loss, dx, dw = ops.linear_cross_entropy_loss_grad(x, w, t)
    z = x.double() @ w[-5:].double().t()
    lse = torch.logsumexp(torch.cat([z, torch.full((4, 1), 0.0, device="cuda", dtype=torch.float64) +
                                     torch.log(torch.tensor(vocab - 5.0, dtype=torch.float64))], 1), 1)
    want = lse - torch.stack([z[0, 4], z[1, 0], z[2, 0] * 0, z[3, 3]])
    # 530000 exponentials in chains of 600, logits of sums of 4096 products in chunks of 1024
    assert ((loss - want).abs() <= 2e-5 * want).all()
    dz = torch.exp(z - lse[:, None])
    dz[0, 4] -= 1
    dz[1, 0] -= 1
    dz[3, 3] -= 1
    ref = dz.t() @ x.double()
    assert ((dw[-5:].double() - ref).norm() / ref.norm()) < 2.0 ** -7
    ref = torch.exp(-lse)[:, None] * x.double()
    assert ((dw[1].double() - ref.sum(0)).norm() / ref.sum(0).norm()) < 2.0 ** -6
    assert torch.isfinite(dx.float()).all()
