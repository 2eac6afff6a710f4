"""Distillation loss from a teacher's top logits, forward and backward, against its formulas in fp64."""
import math

import pytest
import torch

import ops_reference as R

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.bfloat16, torch.float16]
LOWEST = {d: torch.finfo(d).min for d in DT}


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def problem(rows, vocab, top, dtype=torch.float32, tdtype=torch.float32, itype=torch.int32, pad=0, offset=0, seed=0,
            std=2.5):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + rows * 7919 + vocab * 31 + top)
    buf = torch.full((rows * (vocab + pad) + offset + 8,), float("nan"), device="cuda", dtype=dtype)
    z = buf[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    z.copy_(torch.randn(rows, vocab, device="cuda", generator=gen) * std)
    index = torch.rand(rows, vocab, device="cuda", generator=gen).argsort(1)[:, :top].to(itype)
    t = (z.gather(1, index.long()).float() * 0.7 + torch.randn(rows, top, device="cuda", generator=gen) + 3).to(tdtype)
    w = torch.rand(rows, device="cuda", generator=gen) + 0.1
    g = torch.randn(rows, device="cuda", generator=gen)
    return z, t, index, w, g


def check(ops, z, t, index, w, g, T=1.0):
    keep = z.clone()
    loss, lse = ops.distill_forward(z, t, index, temperature=T, row_weight=w)
    rloss, rlse, rd = R.distill(z, t, index, T, w)
    tloss, tlse, td = R.distill_bounds(z, t, index, T, w)
    R.assert_close(lse, rlse, tlse, "lse")
    R.assert_close(loss, rloss, tloss, "loss")
    loss2, d = ops.distill_loss_grad(z, t, index, temperature=T, row_weight=w)
    R.assert_close(loss2, rloss, tloss, "loss of loss_grad")
    assert d.dtype == z.dtype
    R.assert_close(d, rd, td + R.rounding(rd, z.dtype), "dlogits of loss_grad")
    _, _, rd = R.distill(z, t, index, T, w, g)
    _, _, td = R.distill_bounds(z, t, index, T, w, g)
    d2 = ops.distill_backward(g, z, lse, t, index, temperature=T, row_weight=w)
    R.assert_close(d2, rd, td + R.rounding(rd, z.dtype), "dlogits")
    assert torch.equal(z.nan_to_num(), keep.nan_to_num()), "the logits changed"
    # in place of the logits
    z1, z2 = z.clone(), z.clone()
    assert torch.equal(ops.distill_loss_grad(z1, t, index, temperature=T, row_weight=w, out=z1)[1].nan_to_num(),
                       d.nan_to_num())
    ops.distill_backward(g, z2, lse, t, index, temperature=T, row_weight=w, out=z2)
    assert torch.equal(z2.nan_to_num(), d2.nan_to_num())
    return loss, lse, d, d2


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 31, 100, 255, 256, 1000, 1031, 4096, 4099, 32000, 50021, 131072, 262147])
def test_vocabularies(ops, vocab):
    for rows in (1, 3):
        for dtype in DT:
            check(ops, *problem(rows, vocab, min(vocab, 20), dtype), T=1.5)


@pytest.mark.parametrize("rows", [1, 2, 8, 19, 37, 38, 75, 76, 151, 153, 310, 700])
def test_row_counts(ops, rows):
    check(ops, *problem(rows, 2056, 16, torch.bfloat16))
    check(ops, *problem(rows, 12001, 16, torch.float32))


@pytest.mark.parametrize("top", [1, 2, 31, 32, 33, 64, 100, 255, 256, 257, 500, 1024])
def test_tops(ops, top):
    for itype in (torch.int32, torch.int64):
        for tdtype in DT:
            check(ops, *problem(5, 3000, top, torch.bfloat16, tdtype, itype), T=2.0)


@pytest.mark.parametrize("T", [0.05, 0.5, 1.0, 4.0, 100.0])
def test_temperatures(ops, T):
    for dtype in DT:
        check(ops, *problem(6, 5000, 40, dtype), T=T)


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 0), (8, 3), (0, 1), (0, 5), (40, 8)])
def test_strides_and_alignment(ops, pad, offset):
    for vocab in (999, 1024, 40001):
        for dtype in DT:
            check(ops, *problem(7, vocab, 12, dtype, pad=pad, offset=offset))
    # a gradient whose rows start elsewhere than the logits'
    z, t, index, w, g = problem(5, 4100, 9, torch.bfloat16)
    want = ops.distill_loss_grad(z, t, index)[1]
    out = torch.zeros(5 * 4103 + 5, device="cuda", dtype=torch.bfloat16)[3:3 + 5 * 4103].view(5, 4103)[:, :4100]
    assert ops.distill_loss_grad(z, t, index, out=out)[1] is out and torch.equal(out, want)


def test_strided_teacher(ops):
    z, t, index, w, g = problem(6, 800, 40)
    a = check(ops, z, t[:, :17], index[:, :17], w, g)
    b = check(ops, z, t[:, :17].contiguous(), index[:, :17].contiguous(), w, g)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_masked_vocabulary(ops):
    for dtype in DT:
        for low in (-math.inf, LOWEST[dtype]):
            z, t, index, w, g = problem(6, 3001, 10, dtype)
            index = index % 2900
            index = (torch.arange(10, device="cuda") * 290 + index % 290).int()  # distinct, in the real part
            z[:, 2900:] = low
            z[3, :2000] = low
            z.scatter_(1, index.long(), 1.0)
            _, _, d, _ = check(ops, z, t, index, w, g)
            assert not d[:, 2900:].any()


def test_rows_that_a_mask_leaves_empty(ops):
    for dtype in DT:
        # every logit at the type's lowest value: a uniform distribution
        z, t, index, w, g = problem(4, 777, 5, dtype)
        z[1] = LOWEST[dtype]
        loss, lse, d, _ = check(ops, z, t, index, w, g)
        # every logit masked with -inf: there is no distribution, and the row says so; the others do not notice
        clean = ops.distill_loss_grad(z, t, index)
        z[2] = -math.inf
        loss, d = ops.distill_loss_grad(z, t, index)
        keep = torch.tensor([0, 1, 3], device="cuda")
        assert torch.isnan(loss[2]) and torch.isnan(d[2]).any()
        assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(d[keep], clean[1][keep])


def test_teachers_without_entries(ops):
    for dtype in DT:
        z, t, index, w, g = problem(7, 1500, 8, dtype)
        index[1] = -1
        index[2, 3:] = -1
        index[3, 0] = 1500       # just outside
        index[4, 1] = 2 ** 31 - 1
        t[5] = -math.inf
        t[6, :7] = -math.inf
        loss, lse, d, d2 = check(ops, z, t, index, w, g)
        for r in (1, 5):
            assert loss[r] == 0 and not d[r].any() and not d2[r].any()
    z, t, index, w, g = problem(3, 600, 0)
    loss, lse, d, d2 = check(ops, z, t, index, w, g)
    assert not loss.any() and not d.any()
    far = torch.full((3, 2), 2 ** 40 + 1, device="cuda", dtype=torch.int64)  # not truncated to 32 bits
    assert not ops.distill_forward(z, torch.ones(3, 2, device="cuda"), far)[0].any()


def test_teacher_masked_by_the_lowest_value(ops):
    for tdtype in DT:
        z, t, index, w, g = problem(4, 900, 6, torch.bfloat16, tdtype)
        t[0, 2:] = LOWEST[tdtype]
        t[1] = LOWEST[tdtype]  # all alike: uniform over the six
        check(ops, z, t, index, w, g)


def test_repeated_entries(ops):
    for top in (6, 300):
        z, t, index, w, g = problem(5, 3000, top, torch.bfloat16)
        index[0] = index[0, 0]
        index[1, ::2] = index[1, 1]
        check(ops, z, t, index, w, g)


def test_rows_that_do_not_count(ops):
    for dtype in DT:
        z, t, index, w, g = problem(9, 2222, 8, dtype)
        w[::3] = 0
        z[3] = math.nan  # not read
        t[6] = math.nan
        g[1] = 0
        loss, lse, d, d2 = check_counts(ops, z, t, index, w, g)
        for r in (0, 3, 6):
            assert loss[r] == 0 and lse[r] == 0 and not d[r].any() and not d2[r].any()
        assert not d2[1].any() and d[1].any()


def check_counts(ops, z, t, index, w, g):
    loss, lse = ops.distill_forward(z, t, index, row_weight=w)
    rloss, rlse, rd = R.distill(z, t, index, 1.0, w)
    loss2, d = ops.distill_loss_grad(z, t, index, row_weight=w)
    d2 = ops.distill_backward(g, z, lse, t, index, row_weight=w)
    keep = w != 0
    tloss, tlse, td = R.distill_bounds(z[keep], t[keep], index[keep], 1.0, w[keep])
    R.assert_close(loss[keep], rloss[keep], tloss, "loss")
    R.assert_close(lse[keep], rlse[keep], tlse, "lse")
    R.assert_close(d[keep], rd[keep], td + R.rounding(rd[keep], z.dtype), "dlogits")
    assert torch.equal(loss[~keep], loss2[~keep])
    return loss, lse, d, d2


def test_infinite_loss_and_nan(ops):
    z, t, index, w, g = problem(4, 500, 4)
    z[1, index[1, 2].long()] = -math.inf  # the teacher believes in what the student excludes
    z[2, 7] = math.nan
    z[3, 9] = math.inf
    loss, d = ops.distill_loss_grad(z, t, index)
    assert torch.isfinite(loss[0]) and loss[1] == math.inf and torch.isnan(loss[2]) and torch.isnan(loss[3])
    assert torch.isfinite(d[:2]).all() and torch.isnan(d[2]).all()
    rd = R.distill(z[:2], t[:2], index[:2], 1.0)[2]
    td = R.distill_bounds(z[:2], t[:2], index[:2], 1.0)[2]
    R.assert_close(d[:2], rd, td + R.rounding(rd, torch.float32))
    z, t, index, w, g = problem(3, 500, 4)
    t[1, 2] = math.nan
    loss, d = ops.distill_loss_grad(z, t, index)
    assert torch.isnan(loss[1]) and torch.isfinite(loss[[0, 2]]).all() and torch.isfinite(d[[0, 2]]).all()


def test_large_logits(ops):
    z, t, index, w, g = problem(4, 3000, 16, torch.float32, std=1e4)
    check(ops, z, t, index, w, g)
    z, t, index, w, g = problem(4, 3000, 16, torch.bfloat16, std=1e30)
    t = torch.randn_like(t)
    check(ops, z, t, index, w, g, T=2.0)


def test_shapes_and_no_rows(ops):
    z, t, index, w, g = problem(12, 640, 7, torch.bfloat16)
    loss, d = ops.distill_loss_grad(z.view(3, 4, 640), t.view(3, 4, 7), index.view(3, 4, 7), row_weight=w.view(3, 4))
    flat = ops.distill_loss_grad(z, t, index, row_weight=w)
    assert loss.shape == (3, 4) and d.shape == (3, 4, 640)
    assert torch.equal(loss.view(-1), flat[0]) and torch.equal(d.view(12, 640), flat[1])
    one = ops.distill_loss_grad(z[0], t[0], index[0], row_weight=w[0])
    assert one[0].shape == () and torch.equal(one[1], flat[1][0])
    loss, d = ops.distill_loss_grad(z[:0], t[:0], index[:0])
    assert loss.shape == (0,) and d.shape == (0, 640)


@pytest.mark.parametrize("dtype,vocab,pad,offset", [
    (torch.bfloat16, 20000, 0, 0), (torch.bfloat16, 16391, 0, 3), (torch.bfloat16, 110000, 0, 0),
    (torch.float16, 106499, 3, 1), (torch.float32, 9000, 0, 0), (torch.float32, 9001, 2, 1),
    (torch.float32, 50003, 0, 2), (torch.float16, 32768, 8, 0)])
def test_many_long_rows(ops, dtype, vocab, pad, offset):
    rows = 700  # several rows per SM
    z, t, index, w, g = problem(rows, vocab, 50, dtype, pad=pad, offset=offset)
    w[::7] = 0
    w[-3:] = 0.5
    index[5] = -1
    index[11] = index[11, 3]
    z[600, 17:] = -math.inf
    z[600].scatter_(0, index[600].long(), 2.0)
    check(ops, z, t, index, w, g, T=1.5)
    alone = ops.distill_forward(z[333:334], t[333:334], index[333:334], temperature=1.5, row_weight=w[333:334])[0]
    together = ops.distill_loss_grad(z, t, index, temperature=1.5, row_weight=w)
    assert torch.allclose(alone, together[0][333:334], rtol=1e-5)
    first = ops.distill_backward(g, z, torch.zeros_like(w), t, index, row_weight=w)
    assert torch.equal(first, ops.distill_backward(g, z, torch.zeros_like(w), t, index, row_weight=w))


def test_many_long_rows_and_entries(ops):
    z, t, index, w, g = problem(650, 17000, 1024, torch.bfloat16, torch.float16, torch.int64)
    index[3, :] = index[3, 0]
    check(ops, z, t, index, w, g)
    check(ops, z, t[:, :0], index[:, :0], w, g)


@pytest.mark.parametrize("rows,vocab", [(2, 131072), (40, 50021), (400, 8000)])
def test_same_bits_again(ops, rows, vocab):
    z, t, index, w, g = problem(rows, vocab, 64, torch.bfloat16)

    def everything():
        loss, lse = ops.distill_forward(z, t, index, row_weight=w)
        return (loss, lse, ops.distill_backward(g, z, lse, t, index, row_weight=w),
                *ops.distill_loss_grad(z, t, index, row_weight=w))
    first = everything()
    torch.randn(1 << 22, device="cuda").sort()
    assert all(torch.equal(a, b) for a, b in zip(first, everything()))


def test_gradient_against_differences(ops):
    z, t, index, w, g = problem(5, 400, 12)
    for T in (1.0, 3.0):
        d = ops.distill_loss_grad(z, t, index, temperature=T, row_weight=w)[1].double()
        way = torch.randn_like(z).double()
        up, down = (R.distill(z.double() + s * 1e-5 * way, t, index, T, w)[0].sum() for s in (1, -1))
        assert abs((d * way).sum() - (up - down) / 2e-5) <= 1e-5 * (d * way).abs().sum()


def test_other_stream_and_graph(ops):
    z, t, index, w, g = problem(50, 9000, 32, torch.bfloat16)
    loss, d = ops.distill_loss_grad(z, t, index, row_weight=w)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        a, b = ops.distill_loss_grad(z, t, index, row_weight=w, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, loss) and torch.equal(b, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ga, gb = ops.distill_loss_grad(z, t, index, row_weight=w)
    graph.replay()
    assert torch.equal(ga, loss) and torch.equal(gb, d)


def test_autograd(ops):
    z, t, index, w, g = problem(6, 700, 9)
    zz = z.clone().requires_grad_()
    loss = ops.distill_loss(zz, t, index, temperature=2.0, row_weight=w)
    (loss * g).sum().backward()
    _, lse = ops.distill_forward(z, t, index, temperature=2.0, row_weight=w)
    assert torch.equal(zz.grad, ops.distill_backward(g, z, lse, t, index, temperature=2.0, row_weight=w))
    zz.grad = None
    ops.distill_loss(zz, t, index).sum().backward()  # an expanded gradient
    d = ops.distill_loss_grad(z, t, index)[1]
    assert torch.allclose(zz.grad, d, rtol=1e-4, atol=1e-7)


def test_refusals(ops):
    from tensor_grad_clip_gb300 import SomaError
    z, t, index, w, g = problem(4, 100, 5)
    with pytest.raises(TypeError, match="teacher_index"):
        ops.distill_forward(z, t, index.float())
    with pytest.raises(ValueError, match="teacher_index"):
        ops.distill_forward(z, t, index[:, :3])
    with pytest.raises(ValueError, match="teacher_logits"):
        ops.distill_forward(z, t[:3], index)
    with pytest.raises(TypeError, match="row_weight"):
        ops.distill_forward(z, t, index, row_weight=w.half())
    with pytest.raises(SomaError, match="temperature"):
        ops.distill_forward(z, t, index, temperature=0.0)
    with pytest.raises(SomaError, match="top"):
        big = torch.zeros(4, 1025, device="cuda")
        ops.distill_forward(z, big, big.int())
    with pytest.raises(TypeError, match="out"):
        ops.distill_loss_grad(z, t, index, out=z.half())
    with pytest.raises(ValueError, match="lse"):
        ops.distill_backward(g, z, g[:2], t, index)
    with pytest.raises(SomaError, match="vocab"):
        ops.distill_forward(z[:, :0], t, index)
