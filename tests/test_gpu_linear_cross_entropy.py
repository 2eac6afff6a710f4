"""Cross entropy of a linear layer against its formulas in fp64.

Bounds, with u = 2^-24.  A logit is an fp32 sum of k products, whose last bits a tensor core may drop rather than round: off by
at most (k + 8) 2 u sum |x w|.  Its row's log-sum-exp is off
by the largest of those, and by the sum of exponentials: each within 2^-21 of itself, added up in chains of at most 64 + V / 1024
+ 96 additions.  dz is the exponential of a difference, off by what the difference is, and rounded to the type; a gradient
element adds the errors of the dz in its sum, (n + 8) 2 u of the terms' magnitudes and one rounding."""
import math

import pytest
import torch

from ops_reference import HALF_ULP, U32, assert_close, rounding

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def ops():
    from tensor_grad_clip_gb300 import ops
    yield ops
    ops.check(0)


def matrix(rows, cols, dtype, pad=0, offset=0, std=1.0):
    buf = torch.randn(rows * (cols + pad) + offset, device="cuda").mul(std).to(dtype)
    return buf[offset:].view(rows, cols + pad)[:, :cols]


class Case:
    def __init__(self, rows, vocab, k, dtype, xpad=0, wpad=0, offset=0, ignored=0.2, weights=True, scale=1.0):
        self.x = matrix(rows, k, dtype, xpad, offset, 2.0)
        self.w = matrix(vocab, k, dtype, wpad, offset, 1.0 / math.sqrt(k))
        self.t = torch.randint(0, vocab, (rows,), device="cuda")
        out = torch.rand(rows, device="cuda")
        self.t[out < ignored / 3] = -100
        self.t[out > 1 - ignored / 3] = vocab
        self.weight = None
        if weights:
            self.weight = (torch.rand(rows, device="cuda") + 0.5) * scale
            self.weight[(out > 0.5) & (out < 0.5 + ignored / 3)] = 0
        self.g = torch.randn(rows, device="cuda")
        self.rows, self.vocab, self.k, self.dtype = rows, vocab, k, dtype

    def reference(self, grad_loss=None, lse=None, kept=False):
        """Loss, lse, dx, dweight and their bounds in fp64; lse: as given to the backward pass; kept: exponentials are
        rounded to fp16 before dz is, half a step of p, or of fp16's smallest, 2^-24 / 2^14 of the largest (which is at most
        1 above p's own slice: g times 2^-39)."""
        x, w = self.x.double(), self.w.double()
        counts = (self.t >= 0) & (self.t < self.vocab)
        weight = torch.ones(self.rows, device="cuda", dtype=torch.float64) if self.weight is None else self.weight.double()
        counts &= weight != 0
        weight = torch.where(counts, weight, 0.0)
        at = torch.where(counts, self.t, 0)[:, None]
        z = x @ w.t()
        ez = (self.k + 8) * 2 * U32 * (x.abs() @ w.abs().t())
        true = torch.logsumexp(z, 1)
        el = ez.amax(1) + 2.0 ** -21 + (160 + self.vocab / 1024) * U32 + 2 * U32 * true.abs()
        loss = weight * (true - z.gather(1, at)[:, 0])
        e_loss = weight.abs() * (el + ez.gather(1, at)[:, 0] + 4 * U32 * true.abs()) + 2 * U32 * loss.abs()
        r = dict(loss=(torch.where(counts, loss, 0.0), e_loss),
                 lse=(torch.where(counts, true, 0.0), el))
        g = weight if grad_loss is None else torch.where(counts, weight * grad_loss.double(), 0.0)
        used = true if lse is None else torch.where(counts, lse.double(), 0.0)
        p = torch.exp(z - used[:, None])
        dz = p.scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64)) * g[:, None]
        # (a given lse is exact)
        near = ez + (el[:, None] if lse is None else 0.0) + 2 * U32 * (z.abs() + used.abs()[:, None]) + 2.0 ** -21
        e_dz = g.abs()[:, None] * p * torch.expm1(near) + 2 * U32 * (g.abs()[:, None] * p + dz.abs())
        # rounded once to 16 bits; what is scaled below the type's smallest steps (fp16: 2^-25 of 2^14 / the largest |g|)
        step = g.abs().max() * 2.0 ** -38 if self.dtype == torch.float16 else 2.0 ** -126
        if kept:
            e_dz = e_dz + g.abs()[:, None] * (HALF_ULP[torch.float16] * p + 2.0 ** -39)
        e_dz = e_dz + HALF_ULP[self.dtype] * (dz.abs() + e_dz) + step
        mag = dz.abs() + e_dz
        dx, dw = dz @ w, dz.t() @ x
        e_dx = e_dz @ w.abs() + (self.vocab + 20) * 2 * U32 * (mag @ w.abs())
        e_dw = e_dz.t() @ x.abs() + (self.rows + 65) * 2 * U32 * (mag.t() @ x.abs())
        for name, ref, e in (("dx", dx, e_dx), ("dw", dw, e_dw)):
            e = e + rounding(ref.abs() + e, self.dtype)
            if self.dtype == torch.float16:  # 65520 and what is above it round to infinity
                e = torch.where((ref.abs() + e >= 65520) & (ref.abs() - e < 65520), math.inf, e)
                ref = torch.where(ref.abs() - e >= 65520, torch.sign(ref) * math.inf, ref)
            r[name] = (ref, e)
        self.counts = counts
        return r

    def check(self, ops, what=""):
        kw = dict(row_weight=self.weight)
        ref = self.reference(kept=True)
        loss, lse = ops.linear_cross_entropy_forward(self.x, self.w, self.t, **kw)
        assert loss.dtype == lse.dtype == torch.float32
        assert_close(loss, *ref["loss"], f"{what}: loss")
        assert_close(lse, *ref["lse"], f"{what}: lse")
        loss2, dx, dw = ops.linear_cross_entropy_loss_grad(self.x, self.w, self.t, **kw)
        assert torch.equal(loss, loss2), what
        assert dx.dtype == dw.dtype == self.dtype
        assert_close(dx, *ref["dx"], f"{what}: dx")
        assert_close(dw, *ref["dw"], f"{what}: dweight")
        assert not dx[~self.counts].any() and not lse[~self.counts].any()
        ref = self.reference(self.g, lse)
        dx, dw = ops.linear_cross_entropy_backward(self.g, self.x, self.w, self.t, lse, **kw)
        assert_close(dx, *ref["dx"], f"{what}: dx of a gradient")
        assert_close(dw, *ref["dw"], f"{what}: dweight of a gradient")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 5, 63, 64, 65, 128, 129, 300])
def test_small(ops, dtype, rows):
    torch.manual_seed(rows)
    for vocab, k in ((1, 8), (2, 1), (7, 63), (31, 64), (32, 65), (33, 200), (127, 16), (128, 128), (129, 72), (1000, 1003)):
        Case(rows, vocab, k, dtype).check(ops, f"{rows} x {vocab} x {k}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,k", [(1000, 5003, 256), (1024, 5000, 65), (2049, 3001, 520), (255, 40001, 64),
                                          (700, 33000, 40)])
def test_many_tiles(ops, dtype, rows, vocab, k):
    torch.manual_seed(rows)
    Case(rows, vocab, k, dtype).check(ops)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(4096, 70001), (16, 200000)])
def test_pieces_of_the_vocabulary_and_parts_of_the_sum(ops, dtype, rows, vocab):
    torch.manual_seed(1)
    Case(rows, vocab, 64, dtype).check(ops)


def test_a_last_piece_of_one_column(ops):
    """65536 rows take 4096 columns at a time: 16 pieces, the last with one."""
    torch.manual_seed(11)
    rows, vocab, k = 65536, 15 * 4096 + 1, 64
    c = Case(rows, vocab, k, torch.bfloat16)
    c.t[:50] = vocab - 1
    loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)
    dx, dw = ops.linear_cross_entropy_backward(c.g, c.x, c.w, c.t, lse, row_weight=c.weight)
    at = torch.arange(0, rows, 173, device="cuda")
    at[:40] = torch.arange(40, device="cuda")
    part = Case(1, 1, 1, torch.bfloat16)
    part.x, part.w, part.t, part.weight = c.x[at], c.w, c.t[at], c.weight[at]
    part.rows, part.vocab, part.k = len(at), vocab, k
    assert_close(loss[at], *part.reference()["loss"], "loss")
    assert_close(dx[at], *part.reference(c.g[at], lse[at])["dx"], "dx")
    # the last column's gradient, of all rows
    counts = (c.t >= 0) & (c.t < vocab) & (c.weight != 0)
    g = torch.where(counts, c.weight * c.g, 0.0).double()
    z = c.x.double() @ c.w[-1].double()
    dz = g * (torch.exp(z - torch.where(counts, lse, 0.0).double()) - (c.t == vocab - 1).double())
    want = dz @ c.x.double()
    near = 2.0 ** -20 + (k + 8) * 2 * U32 * (c.x.double().abs() @ c.w[-1].double().abs())
    e = g.abs() * 2 * near + 2.0 ** -8 * dz.abs()
    tol = e @ c.x.double().abs() + (rows + 65) * 2 * U32 * (dz.abs() @ c.x.double().abs())
    assert_close(dw[-1], want, tol + rounding(want.abs() + tol, torch.bfloat16), "the last column")
    _, dx2, _ = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, row_weight=c.weight, weight_grad=False)
    assert_close(dx2[at], *part.reference()["dx"], "dx of the loss")


@pytest.mark.parametrize("xpad,wpad,offset", [(0, 0, 1), (3, 0, 0), (8, 8, 0), (0, 5, 0), (1, 1, 3), (8, 0, 4)])
def test_rows_with_gaps_and_odd_starts(ops, xpad, wpad, offset):
    torch.manual_seed(2)
    for k in (64, 100, 129):
        Case(90, 300, k, torch.bfloat16, xpad, wpad, offset).check(ops, f"k {k}")


@pytest.mark.parametrize("scale", [1e-9, 1e-3, 1e4])
def test_gradients_far_from_1(ops, scale):
    """dz is scaled into fp16's range before the products: tiny weights of rows lose nothing in dz."""
    torch.manual_seed(3)
    c = Case(200, 700, 96, torch.bfloat16, scale=scale)
    c.check(ops)
    # fp16 outputs themselves have that range only: compare where they do not underflow
    if scale != 1e-9:
        Case(200, 700, 96, torch.float16, scale=scale if scale > 1 else 1e-3).check(ops)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("powers", [10, 24])
def test_rows_of_very_different_weight(ops, dtype, powers):
    """Each row's own dx, beside rows whose weight is up to 2^powers times as large: bf16 loses nothing, fp16 what lies below
    2^-38 of the largest (half such a step for every dz, in the reference's bound)."""
    torch.manual_seed(14)
    for rows, vocab, k in ((200, 700, 96), (1100, 5000, 64)):
        c = Case(rows, vocab, k, dtype)
        c.weight *= 1024 * torch.exp2(-powers * torch.rand(rows, device="cuda"))
        c.g = torch.sign(c.g)
        c.check(ops)
        ref, bound = c.reference()["dx"]
        if powers == 10:  # no row's bound is set by another's weight: it is below 2^-6 of |g| sum_v p_v |w_v| + |w_t|
            p = torch.softmax(c.x.double() @ c.w.double().t(), 1)
            own = c.weight.double()[:, None] * (p @ c.w.double().abs() + c.w.double().abs()[c.t.clamp(0, vocab - 1)])
            assert (bound <= 2.0 ** -6 * own + 2.0 ** -24)[c.counts].all()


def test_rows_that_do_not_count_reach_nothing(ops):
    torch.manual_seed(4)
    for rows, vocab, k in ((300, 500, 72), (1024, 5000, 64)):
        c = Case(rows, vocab, k, torch.bfloat16, ignored=0.6)
        kw = dict(row_weight=c.weight)
        c.reference()
        loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, **kw)
        clean = (loss, lse, *ops.linear_cross_entropy_backward(c.g, c.x, c.w, c.t, lse, **kw))
        c.x[~c.counts] = math.nan
        c.g[~c.counts] = math.inf
        loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, **kw)
        dirty = (loss, lse, *ops.linear_cross_entropy_backward(c.g, c.x, c.w, c.t, lse, **kw))
        assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
        # and they are only passed over: the others alone give the same losses
        keep = c.counts
        alone, _ = ops.linear_cross_entropy_forward(c.x[keep], c.w, c.t[keep], row_weight=c.weight[keep])
        assert torch.allclose(alone, loss[keep], rtol=1e-5, atol=1e-6)


def test_no_row_counts(ops):
    for rows in (1, 200):
        x, w = matrix(rows, 64, torch.float16), matrix(300, 64, torch.float16)
        t = torch.full((rows,), -1, device="cuda")
        x[0] = math.nan
        loss, dx, dw = ops.linear_cross_entropy_loss_grad(x, w, t)
        assert not loss.any() and not dx.any() and not dw.any()


@pytest.mark.parametrize("rows", [1, 40, 200, 1100])
def test_no_row_counts_and_a_weight_is_not_finite(ops, rows):
    """Every gradient is 0, as where the weight is finite, not 0 times infinity of the padding's logits."""
    x, w = matrix(rows, 64, torch.bfloat16), matrix(3000, 64, torch.bfloat16)
    w[7, 3], w[2999, 60] = math.inf, math.nan
    t = torch.full((rows,), -100, device="cuda")
    loss, dx, dw = ops.linear_cross_entropy_loss_grad(x, w, t)
    assert not loss.any() and not dx.any() and not dw.any()
    one = torch.ones(rows, device="cuda")
    dx, dw = ops.linear_cross_entropy_backward(one, x, w, t, 0 * one)
    assert not dx.any() and not dw.any()


def test_infinities_stay_in_their_row(ops):
    torch.manual_seed(5)
    c = Case(130, 200, 64, torch.bfloat16, ignored=0, weights=False)
    loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t)
    c.x[7, 3], c.x[100, 0] = math.inf, math.nan
    bad = torch.zeros(130, dtype=torch.bool, device="cuda")
    bad[[7, 100]] = True
    loss2, dx, _ = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t)
    assert not torch.isfinite(loss2[bad]).any() and torch.equal(loss2[~bad], loss[~bad])
    assert torch.isfinite(dx[~bad]).all() and not torch.isfinite(dx[bad]).all(1).any()


def test_a_loss_near_0(ops):
    """The target's logit far above all others: the loss is the sum of the others' exponentials."""
    x = torch.zeros(64, 64, dtype=torch.float16, device="cuda")
    w = torch.zeros(1000, 64, dtype=torch.float16, device="cuda")
    w[:64] = torch.eye(64, device="cuda") * 4
    x += torch.eye(64, device="cuda").half() * 4  # logit 16 at its own token, 0 elsewhere
    loss, _ = ops.linear_cross_entropy_forward(x, w, torch.arange(64, device="cuda"))
    want = math.log1p(999 * math.exp(-16))
    # the sum of exponentials, 1.0001, is made in at most 64 additions
    assert abs(loss - want).max() <= 64 * U32 + 1e-6 * want


def test_shapes_and_slices(ops):
    torch.manual_seed(6)
    x, w = matrix(6 * 20, 64, torch.bfloat16).view(6, 20, 64), matrix(90, 64, torch.bfloat16)
    texts = torch.randint(0, 90, (6, 25), device="cuda")
    t = texts[:, 3:23]
    loss, lse = ops.linear_cross_entropy_forward(x, w, t)
    assert loss.shape == lse.shape == (6, 20)
    flat, _ = ops.linear_cross_entropy_forward(x.view(120, 64), w, t.reshape(-1).int())
    assert torch.equal(loss.view(-1), flat)
    loss3, dx, dw = ops.linear_cross_entropy_loss_grad(x, w, t, row_weight=torch.ones(6, 20, device="cuda"))
    assert torch.equal(loss3, loss) and dx.shape == x.shape and dw.shape == w.shape
    for call, first in ((ops.linear_cross_entropy_backward, (torch.ones(6, 20, device="cuda"), x, w, t, lse)),
                        (ops.linear_cross_entropy_loss_grad, (x, w, t))):  # (these round dz once and twice)
        dx, dw = call(*first)[-2:]
        only, none = call(*first, weight_grad=False)[-2:]
        assert none is None and torch.equal(only, dx)
        none, only = call(*first, input_grad=False)[-2:]
        assert none is None and torch.equal(only, dw)
    one, _ = ops.linear_cross_entropy_forward(x[2, 5], w, t[2, 5])
    assert one.shape == ()
    empty, dx, dw = ops.linear_cross_entropy_loss_grad(x[:0], w, t[:0])
    assert empty.shape == (0, 20) and not dw.any()


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_one_target_of_each_text(ops, kind):
    torch.manual_seed(16)
    hidden, w = matrix(6 * 20, 64, torch.bfloat16).view(6, 20, 64), matrix(90, 64, torch.bfloat16)
    texts = torch.randint(-1, 90, (6, 25), device="cuda", dtype=kind)
    x, t = hidden[:, -1], texts[:, 20]
    assert not t.is_contiguous()
    got, want = (ops.linear_cross_entropy_loss_grad(x, w, v) for v in (t, t.contiguous()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    lse = ops.linear_cross_entropy_forward(x, w, t)[1]
    got, want = (ops.linear_cross_entropy_backward(torch.ones(6, device="cuda"), x, w, v, lse) for v in (t, t.contiguous()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_and_differences(ops):
    torch.manual_seed(7)
    c = Case(40, 60, 24, torch.float16, ignored=0.3)
    x, w = c.x.clone().requires_grad_(), c.w.clone().requires_grad_()
    g = torch.randn(40, device="cuda")
    (ops.linear_cross_entropy(x, w, c.t, row_weight=c.weight) * g).sum().backward()
    lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)[1]
    dx, dw = ops.linear_cross_entropy_backward(g, c.x, c.w, c.t, lse, row_weight=c.weight)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)

    def total(x, w):  # the formula in fp64
        z = x @ w.t()
        ok = (c.t >= 0) & (c.t < 60)
        loss = torch.logsumexp(z, 1) - z.gather(1, torch.where(ok, c.t, 0)[:, None])[:, 0]
        return (torch.where(ok & (c.weight != 0), loss * c.weight.double(), 0.0) * g.double()).sum()
    x64, w64, step = c.x.double(), c.w.double(), 1e-5
    for got, where, bound in ((dx, x64, c.reference(g, lse)["dx"][1]), (dw, w64, c.reference(g, lse)["dw"][1])):
        for i, j in ((0, 0), (7, 13), (31, 23)):
            d = torch.zeros_like(where)
            d[i, j] = step
            up, down = (total(x64 + d, w64), total(x64 - d, w64)) if where is x64 else (total(x64, w64 + d), total(x64, w64 - d))
            # a central difference errs by step^2 times the third derivative (below 100 here) and by rounding, 1e-16 / step
            assert abs((up - down).item() / (2 * step) - got[i, j].item()) <= bound[i, j].item() + 1e-7
    expanded = ops.linear_cross_entropy(x, w, c.t)
    x.grad = None
    expanded.sum().backward()
    assert torch.isfinite(x.grad).all()


def test_streams_graphs_and_equal_bits(ops):
    torch.manual_seed(8)
    c = Case(1024, 5000, 128, torch.bfloat16, ignored=0.3)
    kw = dict(row_weight=c.weight)
    want = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, **kw)
    again = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, **kw)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, stream=side, **kw)
    other = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, **kw)  # at once
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(want, got, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, **kw)
    # other rows count in the replay: the graph learns of it on the device
    c.t.copy_(torch.randint(-2000, 5000, (1024,), device="cuda"))
    want = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows", [1, 16, 17])
def test_few_rows_replayed_and_at_once(ops, rows):
    """The last CTA to finish joins few rows: every call and every replay finds its own."""
    torch.manual_seed(10)
    cases = [Case(rows, 20000, 512, torch.bfloat16, ignored=0) for _ in range(2)]
    want = [ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight, stream=s) for c, s in zip(cases, streams)]
           for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    c, graph = cases[0], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        first = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)
        second = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)
    for k in range(5):
        c.t[0] = -1 if k % 2 else 7  # another row counts, or none does
        graph.replay()
        torch.cuda.synchronize()
        loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)
        for g in (first, second):
            assert torch.equal(g[0], loss) and torch.equal(g[1], lse)


def test_the_whole_path_of_a_language_model(ops):
    """Tokens to a step: embedding, layer norm, linear, cross entropy, all gradients, and AdamW with moments in 8 bits."""
    from tensor_grad_clip_gb300 import SomaOpt, TensorList, zeros_8bit
    torch.manual_seed(9)
    vocab, width, rows = 1000, 128, 300
    p = {"table": torch.randn(vocab, width, device="cuda") * 0.05, "gain": torch.ones(width, device="cuda"),
         "shift": torch.zeros(width, device="cuda"), "up": torch.randn(width, width, device="cuda") / math.sqrt(width)}
    tokens, targets = (torch.randint(0, vocab, (rows,), device="cuda") for _ in range(2))
    targets[::7] = -100

    def loss_of(q, f):
        x = f["embedding"](tokens, q["table"], scale=math.sqrt(width))
        h = f["norm"](x, q["gain"], q["shift"])
        y = f["linear"](h, q["up"], x)
        return f["loss"](y, q["table"], targets).sum() / rows
    mine = dict(embedding=ops.embedding, norm=ops.layer_norm, loss=ops.linear_cross_entropy,
                linear=lambda h, w, x: ops.linear(h, w, activation="gelu", residual=x))
    plain = dict(embedding=lambda t, w, scale: w[t] * scale,
                 norm=lambda x, a, b: torch.nn.functional.layer_norm(x, (width,), a, b),
                 linear=lambda h, w, x: torch.nn.functional.gelu(h @ w.t()) + x,
                 loss=lambda y, w, t: torch.nn.functional.cross_entropy(y @ w.t(), t, reduction="none"))
    q = {k: v.bfloat16() if v.dim() == 2 else v.clone() for k, v in p.items()}
    exact = {k: v.double().requires_grad_() for k, v in q.items()}
    q = {k: v.requires_grad_() for k, v in q.items()}
    loss = loss_of(q, mine)
    want = loss_of(exact, plain)
    loss.backward()
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -7 * want.item()
    for k in q:
        off = (q[k].grad.double() - exact[k].grad).norm() / exact[k].grad.norm()
        assert off < 2.0 ** -5, (k, off)  # bf16 activations: a few roundings of 2^-8 in a chain
    names = list(p)
    moments = {k: (zeros_8bit(p[k]), zeros_8bit(p[k])) for k in names}
    opt = SomaOpt(0)
    opt.add_group(lr=1e-2)
    tl = TensorList([p[k] for k in names], [q[k].grad for k in names], [moments[k][0][0] for k in names],
                    [moments[k][1][0] for k in names], groups=[0] * len(names),
                    params_lowp=[q[k].detach() if p[k].dim() == 2 else None for k in names],
                    exp_avg_scales=[moments[k][0][1] for k in names], exp_avg_sq_scales=[moments[k][1][1] for k in names])
    before = {k: p[k].clone() for k in names}
    opt.step(tl, 1.0, 1.0)
    norm = math.sqrt(sum((q[k].grad.double() ** 2).sum().item() for k in names))
    assert math.isclose(opt.get_norm()[0], norm, rel_tol=1e-5)
    for k in names:
        moved = q[k].grad != 0
        # the first step's m / sqrt(v) is the gradient's sign
        sure = moved & (q[k].grad.abs() * min(1.0, 1.0 / norm) > 1e-6)
        assert torch.equal(torch.sign(before[k] - p[k])[sure], torch.sign(q[k].grad.float())[sure]), k


def test_refusals(ops):
    x, w = matrix(8, 32, torch.bfloat16), matrix(50, 32, torch.bfloat16)
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    lse = torch.zeros(8, device="cuda")
    for call, error, word in (
            (lambda: ops.linear_cross_entropy_forward(x.float(), w.float(), t), RuntimeError, "bf16 or fp16"),
            (lambda: ops.linear_cross_entropy_forward(x, w.half(), t), TypeError, "weight"),
            (lambda: ops.linear_cross_entropy_forward(x, w[:, :16], t), ValueError, "weight"),
            (lambda: ops.linear_cross_entropy_forward(x, w, t[:7]), ValueError, "target"),
            (lambda: ops.linear_cross_entropy_forward(x, w, t.float()), TypeError, "target"),
            (lambda: ops.linear_cross_entropy_forward(x, w, t, row_weight=lse[:7]), ValueError, "row_weight"),
            (lambda: ops.linear_cross_entropy_forward(x, w, t, row_weight=lse.double()), TypeError, "row_weight"),
            (lambda: ops.linear_cross_entropy_forward(x, w.t().contiguous().t(), t), ValueError, "unit stride"),
            (lambda: ops.linear_cross_entropy_backward(lse[:7], x, w, t, lse), ValueError, "grad_loss"),
            (lambda: ops.linear_cross_entropy_backward(lse, x, w, t, lse.half()), TypeError, "lse"),
            (lambda: ops.linear_cross_entropy_forward(x.cpu(), w, t), ValueError, "CUDA")):
        with pytest.raises(error, match=word):
            call()


def part_of(c, at):
    """The rows `at` of a case, as a case of their own."""
    part = Case(1, 1, 1, c.dtype)
    part.x, part.w, part.t, part.weight = c.x[at], c.w, c.t[at], None if c.weight is None else c.weight[at]
    part.rows, part.vocab, part.k = len(at), c.vocab, c.k
    return part


@pytest.mark.parametrize("rows,vocab,k", [(65536, 131072, 1024), (65536, 262144, 64), (262144, 131072, 4096), (100, 1 << 25, 8)])
def test_the_workspace_of_the_loss_is_bounded(ops, rows, vocab, k):
    """The rows that count, 36 bytes a row, and 512 MB: not a share of the logits."""
    ops._ops_abi.load()
    pitch = (rows + 255) // 256 * 256
    need = ops._head_bytes(0, False, rows, vocab, k, 1, 1, 0, 0)
    assert need <= pitch * (2 * k + 36) + (512 << 20) + (1 << 20)
    # and with gradients: a piece's dz, an eighth of it, dx in fp32
    both = ops._head_bytes(0, False, rows, vocab, k, 1, 1, 1, 1)
    assert both <= need + max(512 << 20, 512 * pitch, vocab * k * 2) * 9 // 8 + pitch * (k + 255) // 256 * 256 * 4 + (80 << 20)


@pytest.mark.parametrize("rows,vocab,k,some", [(65536, 50021, 64, 300), (1000, 2_200_003, 8, 60), (100, 8_600_001, 8, 20)])
def test_statistics_in_pieces_of_the_vocabulary(ops, rows, vocab, k, some):
    """More than 2^31 logits: their statistics are joined piece by piece."""
    torch.manual_seed(12)
    c = Case(rows, vocab, k, torch.bfloat16)
    loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)
    at = torch.randperm(rows, device="cuda")[:some]
    part = part_of(c, at)
    ref = part.reference()
    assert_close(loss[at], *ref["loss"], "loss")
    assert_close(lse[at], *ref["lse"], "lse")
    again = ops.linear_cross_entropy_forward(c.x, c.w, c.t, row_weight=c.weight)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
    loss2, dx, _ = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, row_weight=c.weight, weight_grad=False)
    assert torch.equal(loss, loss2)
    assert_close(dx[at], *ref["dx"], "dx")


def test_statistics_in_pieces_with_kept_exponentials(ops):
    """As many rows as columns of x are one piece of dz, whose exponentials are kept, but several of statistics."""
    torch.manual_seed(13)
    rows, vocab, k = 16384, 131329, 16384
    c = Case(rows, vocab, k, torch.bfloat16, ignored=0.1)
    kw = dict(row_weight=c.weight)
    loss, lse = ops.linear_cross_entropy_forward(c.x, c.w, c.t, **kw)
    loss2, dx, dw = ops.linear_cross_entropy_loss_grad(c.x, c.w, c.t, **kw)
    assert torch.equal(loss, loss2)
    at = torch.randperm(rows, device="cuda")[:10]
    ref = part_of(c, at).reference(kept=True)
    assert_close(loss[at], *ref["loss"], "loss")
    assert_close(dx[at], *ref["dx"], "dx")
    # the gradients from lse, whose dz is made of the logits: both round dz and the result by 2^-8 at most, at random
    dx1, dw1 = ops.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), c.x, c.w, c.t, lse, **kw)
    for a, b in ((dx, dx1), (dw, dw1)):
        for part in (slice(0, 100), slice(len(a) // 2, len(a) // 2 + 100), slice(len(a) - 100, len(a))):
            assert (a[part].double() - b[part].double()).norm() <= 2.0 ** -6 * b[part].double().norm()


@pytest.mark.parametrize("n,vocab", [(1003, 300000), (4000, 131072), (4096, 131072), (4090, 131073), (257, 1 << 20)])
def test_as_many_rows_as_columns_are_one_piece(ops, n, vocab):
    """The workspace has room for dz of the whole vocabulary: the logits are made once."""
    ops._ops_abi.load()
    need, without = (ops._head_bytes(0, False, n, vocab, n, 1, 1, 0, wanted) for wanted in (1, 0))
    pitch = (n + 255) // 256 * 256
    assert need - without >= pitch * vocab * 2
    # not for one tile of rows more
    more, without = (ops._head_bytes(0, False, pitch + 1, vocab, n, 1, 1, 0, wanted) for wanted in (1, 0))
    if pitch * vocab * 2 >= 512 << 20:
        assert more - without < (pitch + 256) * vocab * 2
