"""Embedding lookup and its gradient against their formulas in fp64.

Bounds: a looked-up element is one fp32 product rounded to the type.  A gradient element is an fp32 sum of n terms (error at
most n units of 2^-24 of the terms' magnitudes, in any order), one fp32 multiply-add and one rounding to the type."""
import math

import pytest
import torch

from ops_reference import U32, assert_close, rounding

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    return ops


def matrix(rows, cols, dtype, pad=0, offset=0, std=1.0):
    buf = torch.randn(rows * (cols + pad) + offset, device="cuda").mul(std).to(dtype)
    return buf[offset:].view(rows, cols + pad)[:, :cols]


def draw_tokens(rows, vocab, kind):
    if kind == "one":
        return torch.full((rows,), vocab - 1, device="cuda")
    if kind == "rising":
        return torch.arange(rows, device="cuda") % vocab
    if kind == "none":
        return torch.full((rows,), -1, device="cuda")
    t = torch.randint(0, vocab, (rows,), device="cuda")
    if kind == "skewed":  # one token in half of the places, some places without one
        t[torch.rand(rows, device="cuda") < 0.5] = vocab // 2
        t[torch.rand(rows, device="cuda") < 0.1] = -1
        t[torch.rand(rows, device="cuda") < 0.1] = vocab
    return t


def reference_backward(dy, index, vocab, scale, out=None):
    """(gradient, sum of its terms' magnitudes, terms) in fp64."""
    keep = (index >= 0) & (index < vocab)
    at, d = index[keep].long(), dy[keep].double() * scale
    ref = torch.zeros(vocab, dy.shape[1], device=dy.device, dtype=torch.float64).index_add_(0, at, d)
    mag = torch.zeros_like(ref).index_add_(0, at, d.abs())
    n = torch.zeros(vocab, 1, device=dy.device, dtype=torch.float64).index_add_(0, at, torch.ones_like(d[:, :1]))
    if out is not None:
        ref, mag = ref + out.double(), mag + out.double().abs()
    return ref, mag, n


def assert_gradient(got, dy, index, vocab, scale, out=None, what=""):
    ref, mag, n = reference_backward(dy, index, vocab, scale, out)
    assert_close(got, ref, (n + 3) * U32 * mag + rounding(ref, got.dtype), what)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols,pad,offset", [(1, 0, 0), (7, 3, 1), (64, 0, 0), (64, 8, 3), (1003, 5, 0), (1032, 0, 0),
                                             (5000, 8, 8)])
def test_lookup(ops, dtype, cols, pad, offset):
    for rows, vocab, scale in ((1, 1, 1.0), (5, 3, 0.5), (300, 1000, math.sqrt(cols)), (2049, 257, -3.7)):
        table = matrix(vocab, cols, dtype, pad, offset)
        for index in (draw_tokens(rows, vocab, "skewed"), draw_tokens(rows, vocab, "rising").int()):
            y = ops.embedding_forward(index, table, scale=scale)
            assert y.dtype == dtype and y.shape == (rows, cols)
            keep = (index >= 0) & (index < vocab)
            ref = table[index.clamp(0, vocab - 1).long()].double() * torch.tensor(scale).float().double()
            ref = ref * keep[:, None]
            assert_close(y, ref, 1.001 * rounding(ref, dtype) + U32 * ref.abs(), f"{rows} x {cols} of {vocab}")
            assert not y[~keep].any()


def test_lookup_keeps_what_the_table_holds(ops):
    table = torch.tensor([[0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, 65504.0, 3.0]], device="cuda")
    y = ops.embedding_forward(torch.zeros(2, dtype=torch.int64, device="cuda"), table)
    assert torch.equal(y.view(torch.int32)[:, [0, 1, 2, 3, 5, 6, 7]], table.view(torch.int32).expand(2, 8)[:, [0, 1, 2, 3, 5, 6, 7]])
    assert torch.isnan(y[:, 4]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["any", "skewed", "one", "rising", "none"])
@pytest.mark.parametrize("rows", [1, 63, 64, 65, 128, 129, 1000, 5003])
def test_gradient(ops, dtype, kind, rows):
    for vocab, cols, pad, offset in ((1, 8, 0, 0), (700, 64, 8, 0), (3000, 137, 2, 1), (70001, 16, 0, 0)):
        index, dy = draw_tokens(rows, vocab, kind), matrix(rows, cols, dtype, pad, offset)
        what = f"{kind}: {rows} rows of {cols}, vocabulary {vocab}"
        got = ops.embedding_backward(dy, index, vocab, scale=0.25)
        assert got.shape == (vocab, cols) and got.dtype == dtype
        assert_gradient(got, dy, index, vocab, 0.25, what=what)
        again = ops.embedding_backward(dy, index.int(), vocab, scale=0.25)
        assert torch.equal(got, again), what


@pytest.mark.parametrize("rows,cols,vocab", [(16384, 1024, 32000), (60000, 72, 131072), (94208, 8, 262143),
                                             (94209, 8, 262144), (300001, 24, 511), (1 << 20, 4, 5_000_000)])
def test_gradient_of_long_batches(ops, rows, cols, vocab):
    for kind in ("skewed", "one"):
        index = draw_tokens(rows, vocab, kind)
        for dtype in (torch.float32, torch.bfloat16):
            dy = matrix(rows, cols, dtype)
            assert_gradient(ops.embedding_backward(dy, index, vocab), dy, index, vocab, 1.0, what=kind)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols,pad", [(64, 0), (1003, 5), (40, 8)])
def test_gradient_added_to_another(ops, dtype, cols, pad):
    vocab, rows = 501, 777
    index, dy = draw_tokens(rows, vocab, "skewed"), matrix(rows, cols, dtype)
    index[:7] = 5
    out = matrix(vocab, cols, dtype, pad)
    whole = out._base
    before, gaps = out.clone(), whole.clone()
    got = ops.embedding_backward(dy, index, vocab, scale=2.0, out=out)
    assert got is out
    assert_gradient(got, dy, index, vocab, 2.0, before)
    hit = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    hit[index[(index >= 0) & (index < vocab)]] = True
    assert torch.equal(out[~hit], before[~hit])
    rest = torch.ones(vocab, cols + pad, dtype=torch.bool, device="cuda")
    rest[:, :cols] = False
    assert torch.equal(whole.view(vocab, cols + pad)[rest], gaps.view(vocab, cols + pad)[rest])


def test_rows_without_a_token_are_not_read(ops):
    index = torch.tensor([3, -1, 3, 99, 1 << 40, -(1 << 40)], device="cuda")
    dy = torch.randn(6, 33, device="cuda")
    dy[[1, 3, 4, 5]] = math.nan
    got = ops.embedding_backward(dy, index, 10)
    assert torch.equal(got[3], dy[0] + dy[2]) and not got[[0, 1, 2, 4, 5, 6, 7, 8, 9]].any()
    assert not ops.embedding_forward(index, dy[:1].expand(10, 33).contiguous())[[1, 3, 4, 5]].any()


def test_infinities_and_nan_stay_with_their_token(ops):
    dy = torch.ones(200, 16, device="cuda")
    index = torch.arange(200, device="cuda") % 5
    dy[7], dy[8, 3] = math.inf, math.nan  # tokens 2 and 3
    got = ops.embedding_backward(dy, index, 6)
    assert torch.isinf(got[2]).all() and torch.isnan(got[3]).sum() == 1
    assert torch.equal(got[[0, 1, 4]], torch.full((3, 16), 40.0, device="cuda"))


def test_no_rows(ops):
    table = torch.randn(9, 12, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert ops.embedding_forward(none, table).shape == (0, 12)
    assert not ops.embedding_backward(torch.zeros(0, 12, device="cuda"), none, 9).any()
    out = table.clone()
    ops.embedding_backward(torch.zeros(0, 12, device="cuda"), none, 9, out=out)
    assert torch.equal(out, table)


def test_a_slice_of_a_batch_of_texts(ops):
    table = torch.randn(100, 24, device="cuda").bfloat16()
    texts = torch.randint(-2, 103, (7, 33), device="cuda")
    inside = texts[:, 2:-5]
    assert not inside.is_contiguous()
    y = ops.embedding_forward(inside, table)
    assert y.shape == (7, 26, 24) and torch.equal(y, ops.embedding_forward(inside.contiguous(), table))
    dy = torch.randn(7, 26, 24, device="cuda").bfloat16()
    assert torch.equal(ops.embedding_backward(dy, inside, 100), ops.embedding_backward(dy, inside.contiguous(), 100))
    one = ops.embedding_forward(texts[3, 4], table)
    assert one.shape == (24,) and torch.equal(one, ops.embedding_forward(texts[3, 4:5], table)[0])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_one_token_of_each_text(ops, kind):
    """A column of a batch of texts, as a generation loop looks it up, and every third token of one text."""
    table = torch.randn(100, 24, device="cuda").bfloat16()
    texts = torch.randint(-2, 103, (70, 33), device="cuda", dtype=kind)
    for index in (texts[:, -1], texts[:, 0], texts[5, ::3], texts[:1, 4], texts[:0, 1]):
        y, whole = ops.embedding_forward(index, table), index.contiguous()
        assert y.shape == (*index.shape, 24) and torch.equal(y, ops.embedding_forward(whole, table))
        dy = torch.randn(len(index), 24, device="cuda").bfloat16()
        assert torch.equal(ops.embedding_backward(dy, index, 100), ops.embedding_backward(dy, whole, 100))
    weight = table.clone().requires_grad_()
    ops.embedding(texts[:, -1], weight).sum().backward()
    assert_gradient(weight.grad, torch.ones(70, 24, device="cuda"), texts[:, -1], 100, 1.0)
    with pytest.raises(ValueError, match="unit stride"):
        ops.embedding_forward(texts[:1, 0].expand(5), table)


def test_autograd_and_differences(ops):
    table = torch.randn(50, 24, device="cuda", requires_grad=True)
    index = torch.randint(-1, 50, (4, 30), device="cuda")
    g = torch.randn(4, 30, 24, device="cuda")
    (ops.embedding(index, table, scale=3.0) * g).sum().backward()
    assert_gradient(table.grad, g.view(120, 24), index.view(-1), 50, 3.0)
    # the loss is linear in the table: differences of any size give the gradient
    with torch.no_grad():
        for v, c in ((index[index >= 0][0].item(), 5), (index[index >= 0][9].item(), 23)):
            step = torch.zeros_like(table)
            step[v, c] = 1.0
            up = (ops.embedding(index, table + step, scale=3.0).double() * g.double()).sum()
            down = (ops.embedding(index, table - step, scale=3.0).double() * g.double()).sum()
            n = int((index == v).sum())
            # table +- 1 and the products round by 2^-24 of values of at most 6 x 3, on both sides
            tol = n * g.abs().max().item() * 4 * 18 * U32 + n * (n + 3) * U32 * 3 * g.abs().max().item()
            assert abs((up - down).item() / 2 - table.grad[v, c].item()) <= tol
    # an expanded gradient
    table.grad = None
    ops.embedding(index, table).sum().backward()
    assert_gradient(table.grad, torch.ones(120, 24, device="cuda"), index.view(-1), 50, 1.0)


def test_streams_and_graphs(ops):
    vocab, index = 4000, torch.randint(0, 4000, (3000,), device="cuda")
    table, dy = matrix(vocab, 256, torch.bfloat16), matrix(3000, 256, torch.bfloat16)
    y, d = ops.embedding_forward(index, table), ops.embedding_backward(dy, index, vocab)
    side = torch.cuda.Stream()
    y2 = ops.embedding_forward(index, table, stream=side)
    d2 = ops.embedding_backward(dy, index, vocab, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(d, d2)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y3 = ops.embedding_forward(index, table)
        d3 = ops.embedding_backward(dy, index, vocab)
        total = ops.embedding_backward(dy, index, vocab, out=d3.clone())
    index.copy_(torch.randint(0, vocab, (3000,), device="cuda"))
    dy.normal_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y3, ops.embedding_forward(index, table))
    assert torch.equal(d3, ops.embedding_backward(dy, index, vocab))
    assert_gradient(total, dy, index, vocab, 1.0, d3)


def test_two_streams_at_once(ops):
    vocab = 20000
    index = torch.randint(0, vocab, (16384,), device="cuda")
    dy = [matrix(16384, 512, torch.bfloat16) for _ in range(2)]
    want = [ops.embedding_backward(d, index, vocab) for d in dy]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[ops.embedding_backward(d, index, vocab, stream=s) for _ in range(4)] for d, s in zip(dy, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)


def test_autograd_is_told_of_out(ops):
    out = torch.zeros(10, 8, device="cuda")
    w = torch.ones(10, 8, device="cuda", requires_grad=True)
    loss = (out * w).sum()
    ops.embedding_backward(torch.ones(3, 8, device="cuda"), torch.tensor([1, 2, 2], device="cuda"), 10, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_refusals(ops):
    table, index = torch.randn(10, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = torch.randn(4, 8, device="cuda")
    with pytest.raises(TypeError, match="index"):
        ops.embedding_forward(index.short(), table)
    with pytest.raises(ValueError, match="dimensions"):
        ops.embedding_forward(index, table[0])
    with pytest.raises(TypeError, match="weight"):
        ops.embedding_forward(index, table.double())
    with pytest.raises(ValueError, match="index"):
        ops.embedding_forward(index.cpu(), table)
    with pytest.raises(ValueError, match="unit stride"):
        ops.embedding_forward(index, table.t())
    with pytest.raises(ValueError, match="dy"):
        ops.embedding_backward(dy[:3], index, 10)
    with pytest.raises(ValueError, match="out"):
        ops.embedding_backward(dy, index, 10, out=table[:9])
    with pytest.raises(TypeError, match="out"):
        ops.embedding_backward(dy, index, 10, out=table.half())
    with pytest.raises(RuntimeError, match="scale"):
        ops.embedding_forward(index, table, scale=math.inf)
    with pytest.raises(RuntimeError, match="vocab"):
        ops.embedding_backward(dy, index, 0, out=table[:0])
