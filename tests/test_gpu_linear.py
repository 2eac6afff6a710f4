"""Linear layer with its epilogue, forward and backward, against its formulas in fp64."""
import itertools

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def matrix(gen, rows, cols, pad, offset, dtype, std=1.0):
    """[rows, cols] N(0, std) inside a buffer of longer rows that starts `offset` elements in; the rest is NaN."""
    buf = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), device="cuda", dtype=dtype)
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.randn(rows, cols, device="cuda", generator=gen) * std)
    return view


def forward(ops, m, n, k, dtype, act="none", bias=True, residual=False, save=False, pad=0, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(m * 7919 + n * 131 + k)
    x, w = matrix(gen, m, k, pad, offset, dtype), matrix(gen, n, k, pad, offset, dtype, k ** -0.5)
    b = torch.randn(n, device="cuda", generator=gen).to(dtype) if bias else None
    res = matrix(gen, m, n, pad, offset, dtype) if residual else None
    got = ops.linear_forward(x, w, b, activation=act, residual=res, save_preactivation=save)
    ry, rz = R.linear_forward(x, w, b, act, res)
    ty, tz = R.linear_forward_bounds(x, w, b, act, res)
    y = got[0] if save else got
    assert y.dtype == dtype and y.is_contiguous()
    R.assert_close(y, ry, ty + R.rounding(ry, dtype), f"y {m}x{n}x{k}")
    if save:
        R.assert_close(got[1], rz, tz + R.rounding(rz, dtype), f"z {m}x{n}x{k}")


def backward(ops, m, n, k, dtype, act="none", pad=0, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(m * 7919 + n * 131 + k + 1)
    x, w = matrix(gen, m, k, pad, offset, dtype), matrix(gen, n, k, pad, offset, dtype, k ** -0.5)
    dy, z = matrix(gen, m, n, pad, offset, dtype), matrix(gen, m, n, pad, offset, dtype)
    keep = [t.clone() for t in (x, w, dy, z)]
    dx, dw, db = ops.linear_backward(dy, x, w, None if act == "none" else z, activation=act)
    refs = R.linear_backward(dy, x, w, z, act)
    tols = R.linear_backward_bounds(dy, x, w, z, act, dtype)
    for name, got, ref, tol in zip(("dx", "dw", "db"), (dx, dw, db), refs, tols):
        assert got.dtype == dtype and got.is_contiguous()
        R.assert_close(got, ref, tol + R.rounding(ref, dtype), f"{name} {m}x{n}x{k}")
    for t, before in zip((x, w, dy, z), keep):
        assert torch.equal(t, before), "an input changed"
    return x, w, dy, z, dx, dw, db


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 3, 5), (7, 64, 64), (1, 128, 1024), (1, 1000, 72), (16, 256, 512), (33, 130, 200),
          (64, 64, 64), (128, 128, 64), (128, 256, 128), (129, 257, 65), (200, 1000, 331), (256, 512, 1024),
          (300, 1016, 264), (1000, 96, 1040), (513, 769, 1025), (1500, 1500, 40), (5, 2000, 3333), (2100, 2300, 520)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward_shapes(ops, m, n, k):
    for dtype in DT:
        forward(ops, m, n, k, dtype)
        forward(ops, m, n, k, dtype, act="gelu", residual=True, save=True)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_backward_shapes(ops, m, n, k):
    for dtype in DT:
        backward(ops, m, n, k, dtype)
        backward(ops, m, n, k, dtype, act="silu")


@pytest.mark.parametrize("m", [1, 2, 3, 4, 8, 15, 16, 17, 31, 32, 48, 63, 64, 65, 96, 127])
def test_few_rows(ops, m):
    for n, k in ((1024, 1024), (520, 2056), (999, 1001), (4096, 512)):
        forward(ops, m, n, k, torch.bfloat16, act="silu", residual=True, save=True)
    backward(ops, m, 1024, 520, torch.float16, act="gelu")
    backward(ops, m, 77, 4097, torch.bfloat16)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual,save", list(itertools.product((False, True), repeat=3)))
def test_epilogues(ops, act, bias, residual, save):
    for m, n, k in ((20, 264, 136), (260, 264, 136), (150, 131, 100)):
        forward(ops, m, n, k, torch.float16, act, bias, residual, save)
        forward(ops, m, n, k, torch.bfloat16, act, bias, residual, save)


@pytest.mark.parametrize("act", ACTS)
def test_activation_gradients(ops, act):
    for m, n, k in ((20, 264, 136), (260, 264, 136), (150, 131, 100)):
        for dtype in DT:
            backward(ops, m, n, k, dtype, act)


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 0), (8, 3), (13, 0), (0, 1), (0, 4), (40, 8)])
def test_strides_and_alignment(ops, pad, offset):
    for m, n, k in ((9, 200, 96), (257, 136, 264), (140, 133, 71)):
        forward(ops, m, n, k, torch.bfloat16, act="relu", residual=True, save=True, pad=pad, offset=offset)
        backward(ops, m, n, k, torch.float16, act="gelu_tanh", pad=pad, offset=offset)


def test_wide_products(ops):
    forward(ops, 700, 4096, 1024, torch.bfloat16, act="gelu", save=True)
    forward(ops, 1300, 1024, 11008, torch.bfloat16, residual=True)
    backward(ops, 900, 4096, 1024, torch.float16, act="gelu")
    forward(ops, 3, 11008, 4096, torch.bfloat16, act="silu")


def test_exact_integers(ops):
    # products and sums of small integers are exact in fp32: so are the results, and so are differences of them
    for m, n, k in ((5, 70, 90), (300, 260, 200), (64, 640, 1000)):
        x = torch.randint(-2, 3, (m, k), device="cuda").bfloat16()
        w = torch.randint(-1, 2, (n, k), device="cuda").bfloat16()
        assert torch.equal(ops.linear_forward(x, w).double(), (x.double() @ w.double().t()).bfloat16().double())
        dy = torch.randint(-1, 2, (m, n), device="cuda").bfloat16()
        dx, dw, db = ops.linear_backward(dy, x, w)
        assert torch.equal(dx.double(), (dy.double() @ w.double()).bfloat16().double())
        assert torch.equal(dw.double(), (dy.double().t() @ x.double()).bfloat16().double())
        assert torch.equal(db.double(), dy.double().sum(0).bfloat16().double())


def test_gradient_against_differences(ops):
    torch.manual_seed(5)
    for act in ACTS[2:]:
        x, w, b, dy = (torch.randn(s, device="cuda").half() for s in ((40, 72), (56, 72), (56,), (40, 56)))
        _, z = ops.linear_forward(x, w, b, activation=act, save_preactivation=True)
        grads = ops.linear_backward(dy, x, w, z, activation=act)
        for k, at in enumerate((x, w, b)):
            d = torch.randn(at.shape, device="cuda").double()
            up, down = ((R.linear_forward(*[t.double() + (s * 1e-5 * d if i == k else 0)
                                            for i, t in enumerate((x, w, b))], act, None)[0] * dy.double()).sum()
                        for s in (1, -1))
            got = (grads[k].double() * d).sum()
            # z, dz and the gradient are each rounded to fp16 (2^-11); z's error moves the slope by less than 1.1 |z| 2^-11,
            # and |z| stays below 40 here
            assert abs(got - (up - down) / 2e-5) <= 2.0 ** -11 * 8 * (grads[k].double().abs() * d.abs()).sum()


def test_infinities_and_nan_stay_in_their_row(ops):
    for m in (4, 200):
        x, w = torch.randn(m, 96, device="cuda").bfloat16(), torch.randn(80, 96, device="cuda").bfloat16()
        clean = ops.linear_forward(x, w)
        for bad in (float("nan"), float("inf")):
            x2 = x.clone()
            x2[2, 5] = bad
            y = ops.linear_forward(x2, w)
            assert not torch.isfinite(y[2]).any()
            keep = torch.arange(m, device="cuda") != 2
            assert torch.equal(y[keep], clean[keep])


def test_some_gradients(ops):
    x, w, dy = (torch.randn(s, device="cuda").half() for s in ((33, 64), (48, 64), (33, 48)))
    z = torch.randn(33, 48, device="cuda").half()
    full = ops.linear_backward(dy, x, w, z, activation="silu")
    for flags in itertools.product((False, True), repeat=3):
        part = ops.linear_backward(dy, x, w, z, activation="silu", input_grad=flags[0], weight_grad=flags[1],
                                   bias_grad=flags[2])
        for want, p, f in zip(flags, part, full):
            assert (p is not None) == want and (not want or torch.equal(p, f))


def test_shapes_and_empty(ops):
    x = torch.randn(2, 3, 5, 40, device="cuda").bfloat16()
    w = torch.randn(24, 40, device="cuda").bfloat16()
    y = ops.linear_forward(x, w)
    assert y.shape == (2, 3, 5, 24)
    assert torch.equal(y.view(-1, 24), ops.linear_forward(x.view(-1, 40), w))
    assert torch.equal(ops.linear_forward(x[0, 0, 0], w), y[0, 0, 0])
    dx, dw, db = ops.linear_backward(y, x, w)
    assert dx.shape == x.shape
    e = x[:0]
    assert ops.linear_forward(e, w).shape == (0, 3, 5, 24)
    dx, dw, db = ops.linear_backward(y[:0], e, w)
    assert dx.shape == e.shape and not dw.any() and not db.any()
    none = w[:0]
    assert ops.linear_forward(x, none).shape == (2, 3, 5, 0)
    dx, dw, db = ops.linear_backward(y[..., :0], x, none)
    assert not dx.any() and dw.shape == (0, 40) and db.shape == (0,)


@pytest.mark.parametrize("m,n,k", [(3, 1024, 2048), (300, 520, 264), (1021, 331, 203)])
def test_same_bits_again(ops, m, n, k):
    first = backward(ops, m, n, k, torch.bfloat16, "gelu")
    x, w, dy, z = first[:4]
    y = ops.linear_forward(x, w, activation="silu")
    for _ in range(3):
        torch.randn(1 << 20, device="cuda").sort()
        again = ops.linear_backward(dy, x, w, z, activation="gelu")
        assert all(torch.equal(a, b) for a, b in zip(again, first[4:]))
        assert torch.equal(y, ops.linear_forward(x, w, activation="silu"))


def test_residual_in_place_through_the_c_abi(ops):
    from tensor_grad_clip_gb300 import _ops_abi as C
    for m, n, k in ((3, 128, 256), (200, 264, 64), (190, 131, 64)):
        x, w = torch.randn(m, k, device="cuda").half(), torch.randn(n, k, device="cuda").half()
        r = torch.randn(m, n, device="cuda").half()
        want = ops.linear_forward(x, w, activation="relu", residual=r)
        assert C.soma_linear_forward(0, x.data_ptr(), k, w.data_ptr(), k, None, r.data_ptr(), n, r.data_ptr(), n, None,
                                     0, None, 0, m, n, k, 2, C.SOMA_ACT_RELU,
                                     torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(r, want)


def test_other_stream_and_graph(ops):
    x, w = torch.randn(300, 520, device="cuda").bfloat16(), torch.randn(264, 520, device="cuda").bfloat16()
    y, z = ops.linear_forward(x, w, activation="gelu", save_preactivation=True)
    grads = ops.linear_backward(y, x, w, z, activation="gelu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.linear_forward(x, w, activation="gelu", stream=side)
    got_b = ops.linear_backward(y, x, w, z, activation="gelu", stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, y) and all(torch.equal(a, c) for a, c in zip(got_b, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gz = ops.linear_forward(x, w, activation="gelu", save_preactivation=True)
        gg = ops.linear_backward(gy, x, w, gz, activation="gelu")
    for _ in range(2):
        graph.replay()
        assert torch.equal(gy, y) and all(torch.equal(a, c) for a, c in zip(gg, grads))


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_autograd(ops, act):
    x, w, b, r = (torch.randn(s, device="cuda").half().requires_grad_() for s in ((3, 20, 64), (48, 64), (48,),
                                                                                  (3, 20, 48)))
    y = ops.linear(x, w, b, activation=act, residual=r)
    y.sum().backward()
    dy = torch.ones(60, 48, device="cuda").half()
    _, z = ops.linear_forward(x.detach().view(60, 64), w.detach(), b.detach(), activation=act, save_preactivation=True)
    dx, dw, db = ops.linear_backward(dy, x.detach().view(60, 64), w.detach(), z, activation=act)
    assert torch.equal(x.grad.view(60, 64), dx) and torch.equal(w.grad, dw) and torch.equal(b.grad, db)
    assert torch.equal(r.grad.view(60, 48), dy)


def test_refusals(ops):
    from tensor_grad_clip_gb300 import SomaError
    x, w = torch.randn(4, 64, device="cuda").half(), torch.randn(8, 64, device="cuda").half()
    y = torch.randn(4, 8, device="cuda").half()
    with pytest.raises(SomaError, match="bf16 or fp16"):
        ops.linear_forward(x.float(), w.float())
    with pytest.raises(ValueError, match="weight: shape"):
        ops.linear_forward(x, w[:, :32])
    with pytest.raises(TypeError, match="weight"):
        ops.linear_forward(x, w.bfloat16())
    with pytest.raises(ValueError, match="unit stride"):
        ops.linear_forward(x, w.t().contiguous().t())
    with pytest.raises(ValueError, match="activation"):
        ops.linear_forward(x, w, activation="tanh")
    with pytest.raises(ValueError, match="residual"):
        ops.linear_forward(x, w, residual=y[:2])
    with pytest.raises(SomaError, match="k must"):
        ops.linear_forward(x[:, :0], w[:, :0])
    with pytest.raises(ValueError, match="preactivation"):
        ops.linear_backward(y, x, w, activation="gelu")
    with pytest.raises(ValueError, match="dy"):
        ops.linear_backward(y[:, :4], x, w)
