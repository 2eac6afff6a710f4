"""Layer norm, forward and backward, against its formulas in fp64."""
import itertools

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def matrix(gen, rows, cols, pad, offset, dtype, std=1.0, mean=0.0):
    """[rows, cols] N(mean, std) inside a buffer of longer rows that starts `offset` elements in; the rest is NaN."""
    buf = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), device="cuda", dtype=dtype)
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.randn(rows, cols, device="cuda", generator=gen) * std + mean)
    return view


def check(ops, rows, cols, dtype, wdtype, pad=0, offset=0, affine=True, eps=1e-5, std=1.0, mean=0.0, x=None, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + rows * 131 + cols)
    if x is None:
        x = matrix(gen, rows, cols, pad, offset, dtype, std, mean)
    dy = matrix(gen, rows, cols, pad, offset, dtype)
    w = b = None
    if affine:
        w = (torch.randn(cols, device="cuda", generator=gen) * 0.3 + 1).to(wdtype)
        b = torch.randn(cols, device="cuda", generator=gen).to(wdtype)
    keep_x, keep_dy = x.clone(), dy.clone()
    y, mu, rstd = ops.layer_norm_forward(x, w, b, eps=eps)
    assert y.dtype == dtype and mu.dtype == rstd.dtype == torch.float32
    ry, rmu, rrstd = R.norm_forward(x, w, b, eps)
    ty, tmu, trstd = R.norm_forward_bounds(x, w, b, eps, ry, rmu, rrstd)
    R.assert_close(mu, rmu, tmu, "mean")
    R.assert_close(rstd, rrstd, trstd, "rstd")
    R.assert_close(y, ry, ty + R.rounding(ry, dtype), "y")
    weight = w if w is not None else torch.ones(cols, device="cuda", dtype=wdtype)
    dx, dw, db = ops.layer_norm_backward(dy, x, weight, mu, rstd)
    rdx, rdw, rdb = R.norm_backward(dy, x, w, mu, rstd)
    tdx, tdw, tdb = R.norm_backward_bounds(dy, x, w, mu, rstd)
    assert dx.dtype == dtype and dw.dtype == db.dtype == wdtype
    R.assert_close(dx, rdx, tdx + R.rounding(rdx, dtype), "dx")
    R.assert_close(dw, rdw, tdw + R.rounding(rdw, wdtype), "dweight")
    R.assert_close(db, rdb, tdb + R.rounding(rdb, wdtype), "dbias")
    assert torch.equal(x, keep_x) and torch.equal(dy, keep_dy), "an input changed"
    return y, mu, rstd, dx, dw, db


@pytest.mark.parametrize("cols", [1, 2, 7, 8, 31, 33, 64, 100, 255, 256, 264, 513, 1000, 1024, 1031, 2048, 4096, 4099,
                                  8192, 8200, 11008, 16384, 16391, 40003])
def test_widths(ops, cols):
    for rows, dtype in itertools.product((1, 3, 37), DT):
        check(ops, rows, cols, dtype, torch.float32)


@pytest.mark.parametrize("rows", [1, 2, 5, 16, 151, 153, 609, 2500])
@pytest.mark.parametrize("dtype", DT)
def test_row_counts(ops, rows, dtype):
    check(ops, rows, 520, dtype, dtype)
    check(ops, rows, 1024, dtype, torch.float32)


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 0), (8, 3), (13, 0), (0, 1), (0, 5), (40, 8)])
@pytest.mark.parametrize("dtype", DT)
def test_strides_and_alignment(ops, pad, offset, dtype):
    for cols in (97, 128, 1024, 4099, 20000):
        check(ops, 21, cols, dtype, dtype, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", DT)
def test_without_weight_and_bias(ops, dtype):
    check(ops, 9, 777, dtype, dtype, affine=False)
    x = torch.randn(9, 64, device="cuda", dtype=dtype)
    w = torch.rand(64, device="cuda").to(dtype)
    y, mu, rstd = ops.layer_norm_forward(x, w)
    assert torch.equal(y, ops.layer_norm_forward(x, w, torch.zeros_like(w))[0])
    dx, dw, db = ops.layer_norm_backward(y, x, None, mu, rstd)
    assert dw is None and db is None
    assert torch.equal(dx, ops.layer_norm_backward(y, x, torch.ones_like(w), mu, rstd)[0])
    full = ops.layer_norm_backward(y, x, w, mu, rstd)
    for flags in itertools.product((False, True), repeat=3):
        part = ops.layer_norm_backward(y, x, w, mu, rstd, input_grad=flags[0], weight_grad=flags[1],
                                       bias_grad=flags[2])
        for want, p, f in zip(flags, part, full):
            assert (p is not None) == want and (not want or torch.equal(p, f))


def test_large_mean_and_scale(ops):
    check(ops, 11, 4096, torch.float32, torch.float32, mean=1000.0)
    check(ops, 11, 4096, torch.float32, torch.float32, std=1e15)
    check(ops, 11, 1000, torch.float32, torch.float32, std=1e-12)
    check(ops, 11, 1000, torch.bfloat16, torch.float32, std=1e-3, mean=2.0)


def test_constant_rows_and_special_values(ops):
    x = torch.full((4, 1024), 3.0, device="cuda")
    y, mu, rstd = ops.layer_norm_forward(x, eps=1e-5)
    assert torch.equal(y, torch.zeros_like(y)) and torch.equal(mu, x[:, 0])
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    # a NaN or an infinity stays in its own row
    for bad in (float("nan"), float("inf"), -float("inf")):
        for cols in (40, 4096, 4099, 40000):
            x = torch.randn(5, cols, device="cuda")
            clean = ops.layer_norm_forward(x)[0]
            x[2, cols // 3] = bad
            y, mu, rstd = ops.layer_norm_forward(x)
            assert torch.isnan(y[2]).all() and torch.isnan(rstd[2])
            keep = torch.arange(5, device="cuda") != 2
            assert torch.equal(y[keep], clean[keep])


def test_shapes(ops):
    x = torch.randn(3, 5, 7, 48, device="cuda", dtype=torch.bfloat16)
    w, b = torch.rand(48, device="cuda"), torch.rand(48, device="cuda")
    y, mu, rstd = ops.layer_norm_forward(x, w, b)
    flat = ops.layer_norm_forward(x.view(-1, 48), w, b)
    assert y.shape == x.shape and torch.equal(y.view(-1, 48), flat[0]) and mu.shape == (105,)
    dx, dw, db = ops.layer_norm_backward(y, x, w, mu, rstd)
    assert dx.shape == x.shape
    y1, mu1, _ = ops.layer_norm_forward(x[0, 0, 0], w, b)
    assert y1.shape == (48,) and torch.equal(y1, y[0, 0, 0])
    # padded rows in three dimensions
    wide = torch.randn(3, 5, 50, device="cuda")
    z = ops.layer_norm_forward(wide[..., :48], w, b)[0]
    assert z.shape == (3, 5, 48)
    assert torch.equal(z, ops.layer_norm_forward(wide[..., :48].contiguous(), w, b)[0])


@pytest.mark.parametrize("cols", [64, 4099])
def test_no_rows(ops, cols):
    x = torch.empty(0, cols, device="cuda")
    w = torch.ones(cols, device="cuda")
    y, mu, rstd = ops.layer_norm_forward(x, w, w)
    assert y.shape == (0, cols) and mu.numel() == 0
    dx, dw, db = ops.layer_norm_backward(x, x, w, mu, rstd)
    assert dx.shape == (0, cols) and not dw.any() and not db.any()


@pytest.mark.parametrize("rows,cols", [(700, 1024), (300, 4099), (64, 16384)])
def test_same_bits_again_and_after_other_work(ops, rows, cols):
    x, dy = (torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w, b = torch.rand(cols, device="cuda"), torch.rand(cols, device="cuda")

    def both():
        y, mu, rstd = ops.layer_norm_forward(x, w, b)
        return (y, mu, rstd, *ops.layer_norm_backward(dy, x, w, mu, rstd))
    first = both()
    torch.randn(1 << 22, device="cuda").sort()
    for a, c in zip(first, both()):
        assert torch.equal(a, c)


def test_in_place_through_the_c_abi(ops):
    from tensor_grad_clip_gb300 import _ops_abi as C
    for cols in (96, 1024, 4099, 40000):
        x = torch.randn(17, cols, device="cuda", dtype=torch.float16)
        dy = torch.randn_like(x)
        y, mu, rstd = ops.layer_norm_forward(x)
        dx = ops.layer_norm_backward(dy, x, None, mu, rstd)[0]
        s = torch.cuda.current_stream().cuda_stream
        for target in (x.clone(), dy.clone()):
            same_x = target.data_ptr() if torch.equal(target, x) else x.data_ptr()
            same_dy = target.data_ptr() if torch.equal(target, dy) else dy.data_ptr()
            assert C.soma_layer_norm_backward(0, same_dy, cols, same_x, cols, None, mu.data_ptr(), rstd.data_ptr(),
                                              target.data_ptr(), cols, None, None, None, 0, 17, cols, 2, 2, s) == 0
            assert torch.equal(target, dx)
        t = x.clone()
        assert C.soma_layer_norm_forward(0, t.data_ptr(), cols, None, None, t.data_ptr(), cols, None, None, 17, cols,
                                         2, 2, 1e-5, s) == 0
        assert torch.equal(t, y)


def test_other_stream_and_graph(ops):
    x = torch.randn(500, 2048, device="cuda")
    w, b = torch.rand(2048, device="cuda"), torch.rand(2048, device="cuda")
    y, mu, rstd = ops.layer_norm_forward(x, w, b)
    grads = ops.layer_norm_backward(y, x, w, mu, rstd)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = ops.layer_norm_forward(x, w, b, stream=stream)
        got_b = ops.layer_norm_backward(got[0], x, w, got[1], got[2], stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], y) and all(torch.equal(a, c) for a, c in zip(got_b, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gmu, grstd = ops.layer_norm_forward(x, w, b)
        ggrads = ops.layer_norm_backward(gy, x, w, gmu, grstd)
    for _ in range(2):
        graph.replay()
        assert torch.equal(gy, y) and all(torch.equal(a, c) for a, c in zip(ggrads, grads))


def test_gradient_against_differences(ops):
    torch.manual_seed(3)
    x, w, b, dy = (torch.randn(n, device="cuda") for n in ((6, 300), 300, 300, (6, 300)))
    _, mu, rstd = ops.layer_norm_forward(x, w, b)
    grads = ops.layer_norm_backward(dy, x, w, mu, rstd)
    for k, at in enumerate((x, w, b)):
        d = torch.randn_like(at).double()
        args = [[t.double() + (s * 1e-5 * d if i == k else 0) for i, t in enumerate((x, w, b))] for s in (1, -1)]
        up, down = ((R.norm_forward(*a, 1e-5)[0] * dy).sum() for a in args)
        slope = (up - down) / 2e-5
        got = (grads[k].double() * d).sum()
        # fp64 central difference: good to about 1e-9; the gradient to a few fp32 units of its terms
        assert abs(got - slope) <= 1e-5 * (grads[k].double() * d).abs().sum()


@pytest.mark.parametrize("affine", ["both", "weight", "bias", "none"])
def test_autograd(ops, affine):
    x = torch.randn(4, 10, 96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    w = torch.rand(96, device="cuda", requires_grad=True) if affine in ("both", "weight") else None
    b = torch.rand(96, device="cuda", requires_grad=True) if affine in ("both", "bias") else None
    y = ops.layer_norm(x, w, b)
    y.sum().backward()  # an expanded gradient
    _, mu, rstd = ops.layer_norm_forward(x.detach(), w, b)
    rdx, rdw, rdb = R.norm_backward(torch.ones(40, 96, device="cuda"), x.detach().view(40, 96), w, mu, rstd)
    tdx, tdw, tdb = R.norm_backward_bounds(torch.ones(40, 96, device="cuda"), x.detach().view(40, 96), w, mu, rstd)
    R.assert_close(x.grad.view(40, 96), rdx, tdx + R.rounding(rdx, torch.bfloat16), "dx")
    if w is not None:
        R.assert_close(w.grad, rdw, tdw, "dweight")
    if b is not None:
        R.assert_close(b.grad, rdb, tdb, "dbias")


def test_refusals(ops):
    from tensor_grad_clip_gb300 import SomaError
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    mu, rstd = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="unit stride"):
        ops.layer_norm_forward(x.t())
    with pytest.raises(ValueError, match="evenly spaced"):
        ops.layer_norm_forward(torch.randn(4, 6, 64, device="cuda")[:, ::2][:, :2].transpose(0, 1))
    with pytest.raises(ValueError, match="weight: shape"):
        ops.layer_norm_forward(x, w[:32])
    with pytest.raises(TypeError, match="bias"):
        ops.layer_norm_forward(x, w, w.half())
    with pytest.raises(TypeError, match="float64"):
        ops.layer_norm_forward(x.double())
    with pytest.raises(SomaError, match="param_dtype"):
        ops.layer_norm_forward(x, w.half(), w.half())
    with pytest.raises(SomaError, match="eps"):
        ops.layer_norm_forward(x, w, w, eps=-1.0)
    with pytest.raises(SomaError, match="stride"):
        ops.layer_norm_forward(x[:1].expand(4, 64))
    with pytest.raises(SomaError, match="cols"):
        ops.layer_norm_forward(x[:, :0])
    with pytest.raises(TypeError, match="dy"):
        ops.layer_norm_backward(x.half(), x, w, mu, rstd)
    with pytest.raises(ValueError, match="mean"):
        ops.layer_norm_backward(x, x, w, mu[:3], rstd)
    with pytest.raises(ValueError, match="CUDA"):
        ops.layer_norm_forward(x.cpu())
