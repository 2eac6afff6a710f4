"""The optimizer step with moments in 8 bits against its formulas in fp64.

Bounds: with u = 2^-24, m, v and p each take a handful of fp32 operations, every one off by at most u of its result; a sum of
two terms errs by u of the larger magnitude.  A code is the one that the definition gives in fp64, except where the element is
so near to the border between two codes that fp32 cannot tell; there it is the neighbour."""
import math

import pytest
import torch

from ops_reference import U32
from tensor_grad_clip_gb300 import SomaOpt, TensorList, from_8bit, to_8bit, zeros_8bit

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BLOCK = 256
HP = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)


def chance(index, step):
    """32 bits of the element with this index in its tensor, at this step."""
    low = 0xffffffff
    x = (index & low) ^ (((index >> 32) * 0xc4a8b3f7 + step * 0x9e3779b9) & low)
    x = ((x ^ (x >> 16)) * 0x49a901a7) & low
    x = ((x ^ (x >> 15)) * 0x5fe29a0f) & low
    return x ^ (x >> 16)


class Entry:
    """One tensor of a list, its parts at odd places of larger buffers where `shift` says so."""

    def __init__(self, n, grad=torch.float32, copy=None, shift=0, eight=True, std=1.0, quiet=False):
        def buffer(dtype, by):
            raw = torch.zeros(n + 16 + by, dtype=torch.uint8 if dtype == F8 else dtype, device="cuda")
            return raw, (raw.view(F8) if dtype == F8 else raw)[8 + by:8 + by + n]
        self.n, self.eight = n, eight
        self.buffers = []

        def make(dtype, by, value):
            raw, view = buffer(dtype, by)
            view.copy_(value)
            self.buffers.append((raw, view))
            return view
        by = shift
        self.p = make(torch.float32, by, torch.randn(n, device="cuda") * 0.02)
        self.g = make(grad, by, torch.randn(n, device="cuda") * (0.0 if quiet else std))
        self.copy = None if copy is None else make(copy, by, torch.zeros(n, device="cuda"))
        scale = torch.exp(torch.randn(-(-n // BLOCK), device="cuda")).repeat_interleave(BLOCK)[:n]
        m, root = torch.randn(n, device="cuda") * scale * 1e-3, torch.randn(n, device="cuda").abs() * scale * 3e-3
        if eight:
            (mc, self.ms), (vc, self.vs) = to_8bit(m), to_8bit(root)
            self.m, self.v = make(F8, by, mc), make(F8, by, vc)
        else:
            self.m, self.v, self.ms, self.vs = make(torch.float32, by, m), make(torch.float32, by, root ** 2), None, None
        self.guards = [raw.clone() for raw, _ in self.buffers]

    def moments(self):
        """(m, sqrt(v)) in fp64."""
        if not self.eight:
            return self.m.double(), self.v.double().sqrt()
        wide = [s.double().repeat_interleave(BLOCK)[:self.n] for s in (self.ms, self.vs)]
        return self.m.double() * wide[0], self.v.double() * wide[1]

    def only_views_changed(self):
        for (raw, view), before in zip(self.buffers, self.guards):
            outside = torch.ones(raw.numel(), dtype=torch.bool, device="cuda")
            at = view.storage_offset()
            outside[at:at + self.n] = False
            assert torch.equal(raw.view(before.dtype)[outside], before[outside])


def make_list(entries, groups=None, **kw):
    return TensorList([e.p for e in entries], [e.g for e in entries], [e.m for e in entries], [e.v for e in entries],
                      groups=groups or [0] * len(entries), params_lowp=[e.copy for e in entries],
                      exp_avg_scales=[e.ms for e in entries], exp_avg_sq_scales=[e.vs for e in entries], **kw)


def gap_of(y):
    """Distance between e4m3 neighbours around y >= 0."""
    return torch.exp2(torch.frexp(y.clamp(min=2.0 ** -6)).exponent.double() - 4)


def check_codes(got_codes, got_scales, x, err, bits, least, what):
    """Codes and scales of the fp64 values x, each known to within err."""
    n = x.numel()
    pad = (0, -n % BLOCK)
    blocks = torch.nn.functional.pad(x.abs(), pad).view(-1, BLOCK)
    top = blocks.amax(1)
    top_err = torch.nn.functional.pad(err, pad).view(-1, BLOCK).amax(1)
    assert ((got_scales.double() - top / 448).abs() <= top_err / 448 + 2 * U32 * top / 448).all(), f"{what}: scales"
    top, top_err = (t.repeat_interleave(BLOCK)[:n] for t in (top, top_err))
    live = top > 0
    per = torch.where(live, 448 / torch.where(live, top, 1.0), 0.0)
    y = x.abs() * per
    # |x| (448 / top): two roundings, and what x and top are off themselves
    off = err * per + y * (3 * U32 + torch.where(live, top_err / torch.where(live, top, 1.0), 0.0))
    gap = gap_of(y)
    place = y / gap + (bits.double() + 0.5) / 65536
    want = torch.floor(place) * gap
    if least:
        want = torch.where(y > 0, want.clamp(min=2.0 ** -9), want)
    want = want.clamp(max=448)
    got = got_codes.double().abs()
    near = (place - place.round()).abs() <= off / gap + 2.0 ** -20
    wrong = (got != want) & ~near
    assert not wrong.any(), f"{what}: {int(wrong.sum())} codes of {n}, first at {int(wrong.nonzero()[0])}"
    assert ((got - want).abs() <= 2 * gap).all(), f"{what}: a code that is no neighbour"
    # (the check says something: off / gap is 1e-5 for most elements, so about that share of them; one whose two terms
    # cancel is known worse, and in a tensor of a few elements one is a large share)
    assert near.sum() <= 3 + n / 1000, f"{what}: too many codes that fp32 cannot tell"
    assert (torch.sign(got_codes.double()) * torch.sign(x) >= 0).all()


def reference_step(entries, t, hp, divisor, max_norm, scales_of=None):
    """(p, m, sqrt(v), their errors) of each entry in fp64, from the entries as they are."""
    norm = math.sqrt(sum((e.g.double() ** 2).sum().item() for e in entries)) / divisor
    c = min(1.0, max_norm / (norm + 1e-6))
    b1, b2 = hp["betas"]
    out = []
    for e in entries:
        x = e.g.double() * (c / divisor)
        m0, r0 = e.moments()
        m = b1 * m0 + (1 - b1) * x
        v = b2 * r0 ** 2 + (1 - b2) * x ** 2
        r = v.sqrt()
        # the scale is off by 2^-22 or so (an fp32 sum of squares); constants, products and sums by u each
        em = 8 * U32 * (b1 * m0.abs() + (1 - b1) * x.abs())
        er = 8 * U32 * r
        denominator = r / math.sqrt(1 - b2 ** t) + hp["eps"]
        step = hp["lr"] / (1 - b1 ** t) * m / denominator
        p = e.p.double() * (1 - hp["lr"] * hp["weight_decay"]) - step
        ep = 4 * U32 * e.p.double().abs() + 24 * U32 * step.abs() + hp["lr"] / (1 - b1 ** t) * em / denominator
        out.append((p, m, r, ep, em, er))
    return norm, c, out


def check_step(entries, t, want, what=""):
    for k, (e, (p, m, r, ep, em, er)) in enumerate(zip(entries, want)):
        name = f"{what} entry {k} of {e.n}"
        assert ((e.p.double() - p).abs() <= ep).all(), f"{name}: weights"
        if e.copy is not None:
            assert torch.equal(e.copy, e.p.to(e.copy.dtype)), f"{name}: copy"
        if e.eight:
            bits = chance(torch.arange(e.n, device="cuda"), t)
            check_codes(e.m, e.ms, m, em, bits & 0xffff, False, f"{name}: m")
            check_codes(e.v, e.vs, r, er, bits >> 16, True, f"{name}: v")
        else:
            assert ((e.m.double() - m).abs() <= em).all(), f"{name}: m"
            assert ((e.v.double() - r ** 2).abs() <= 2 * r * er).all(), f"{name}: v"
        e.only_views_changed()


def new_opt(step=0, **kw):
    opt = SomaOpt(0)
    opt.add_group(**{**HP, **kw})
    opt.set_group_step(0, step)
    return opt


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("copy", [None, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shift", [0, 1, 4, 5])
def test_a_step(grad, copy, shift):
    torch.manual_seed(1)
    entries = [Entry(n, grad, copy, shift) for n in (1, 7, 8, 255, 256, 257, 1000, 2048, 8191, 8192, 8193, 70001)]
    opt = new_opt(step=9)
    want = reference_step(entries, 10, HP, 4.0, 1.0)
    opt.step(make_list(entries), 4.0, 1.0)
    norm, c, bad = opt.get_norm()
    assert math.isclose(norm, want[0], rel_tol=1e-5) and math.isclose(c, want[1], rel_tol=1e-5) and not bad
    check_step(entries, 10, want[2])
    assert opt.get_group_step(0) == 10 and opt.plan()["launches_per_step"] == 2


@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_entries_of_both_kinds_and_many_steps(max_norm):
    torch.manual_seed(2)
    entries = [Entry(3000 + 77 * k, (torch.float32, torch.bfloat16)[k % 2], eight=k % 3 != 0, quiet=k == 4)
               for k in range(9)]
    opt, tl = new_opt(), make_list(entries)
    for t in range(1, 6):
        for e in entries:
            e.g.mul_(0.9)
            e.guards[1] = e.buffers[1][0].clone()
        want = reference_step(entries, t, HP, 8.0, max_norm)
        opt.step(tl, 8.0, max_norm)
        check_step(entries, t, want[2], f"step {t}")
    assert opt.plan()["launches_per_step"] == 3
    assert opt.cache_stats()["builds"] == 1


def test_many_small_tensors():
    torch.manual_seed(3)
    entries = [Entry(1 + 37 * k % 900, eight=k % 5 != 0) for k in range(700)]
    opt = new_opt(step=99)
    want = reference_step(entries, 100, HP, 1.0, 1.0)
    opt.step(make_list(entries), 1.0, 1.0)
    check_step(entries, 100, want[2])


def test_from_zeros():
    torch.manual_seed(4)
    e = Entry(5000, torch.bfloat16)
    (m, e.ms), (v, e.vs) = zeros_8bit(e.p), zeros_8bit(e.p)
    e.m.copy_(m), e.v.copy_(v)
    opt = new_opt()
    want = reference_step([e], 1, HP, 1.0, 1.0)
    opt.step(make_list([e]), 1.0, 1.0)
    check_step([e], 1, want[2])


def test_frozen_empty_and_unowned_entries():
    torch.manual_seed(5)
    entries = [Entry(600) for _ in range(4)]
    empty = Entry(1)
    empty.n = 0
    for name in ("p", "g", "m", "v", "ms", "vs"):
        setattr(empty, name, getattr(empty, name)[:0])
    before = [x.clone() for x in (entries[0].p, entries[0].m.view(torch.uint8), entries[0].ms)]
    opt = new_opt()
    tl = make_list(entries + [empty], trainable=[False, True, True, True, True], owned=[True, True, False, True, True])
    want = reference_step([entries[1], entries[3]], 1, HP, 1.0, 1.0)
    opt.step(tl, 1.0, 1.0)
    assert math.isclose(opt.get_norm()[0], want[0], rel_tol=1e-5)
    check_step([entries[1], entries[3]], 1, want[2])
    after = (entries[0].p, entries[0].m.view(torch.uint8), entries[0].ms)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    entries[0].only_views_changed()


def clones(entries):
    return [[x.clone() if x is not None else None for x in (e.p, e.m.view(torch.uint8), e.v.view(torch.uint8), e.ms, e.vs)]
            for e in entries]


def put_back(entries, saved):
    for e, (p, m, v, ms, vs) in zip(entries, saved):
        e.p.copy_(p), e.m.view(torch.uint8).copy_(m), e.v.view(torch.uint8).copy_(v)
        if ms is not None:
            e.ms.copy_(ms), e.vs.copy_(vs)


def same(a, b):
    return all(x is y or torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


@pytest.mark.parametrize("own_divisor", [False, True])
def test_the_same_bits_on_every_path(own_divisor):
    """Regular, repeated, captured and multi-rank steps, and a run resumed from a checkpoint."""
    torch.manual_seed(6)
    entries = [Entry(4000 + 300 * k, torch.bfloat16, eight=k != 2) for k in range(5)]
    groups = [0, 1, 0, 1, 1]
    start = clones(entries)

    def fresh():
        opt = SomaOpt(0)
        opt.add_group(**HP)
        opt.add_group(**{**HP, "weight_decay": 0.0, "lr": 3e-4})
        opt.set_group_step(1, 40)
        if own_divisor:
            opt.set_group_divisor(1, 16.0)
        put_back(entries, start)
        return opt, make_list(entries, groups)
    opt, tl = fresh()
    results = []
    for _ in range(3):
        opt.step(tl, 8.0, 0.5)
        results.append(clones(entries))
    opt, tl = fresh()
    for k in range(3):
        opt.step(tl, 8.0, 0.5)
        assert same(results[k], clones(entries))
        if k == 1:
            other = SomaOpt(0)
            other.load_state_dict(opt.state_dict())
            opt = other
    # captured
    opt, tl = fresh()
    opt.push_groups()
    opt.step_graph(tl, 8.0, 0.5)
    assert same(results[0], clones(entries))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step_graph(tl, 8.0, 0.5)
    for k in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        assert same(results[k], clones(entries))
    opt.pull_groups()
    assert opt.get_group_step(0) == 3 and opt.get_group_step(1) == 43
    # in two halves
    opt, tl = fresh()
    sums = torch.zeros(1, dtype=torch.float64, device="cuda")
    opt.sumsq(tl, 8.0, sums)
    opt.step_from_sumsq(tl, 8.0, 0.5, sums)
    want = results[0]
    for (p, m, v, ms, vs), (q, *_) in zip(clones(entries), want):
        assert torch.allclose(p, q, rtol=1e-6, atol=1e-9)
    assert opt.cache_stats()["builds"] == 1


def test_rounding_keeps_the_mean():
    """200 steps without gradients: every step moves sqrt(v) by 0.05 % and m by 10 %, which e4m3 alone could not follow."""
    torch.manual_seed(7)
    n, steps = 1 << 18, 200
    e = Entry(n, quiet=True)
    e.g.zero_()
    root = torch.rand(n, device="cuda") + 0.5
    # one large element in each block sets its scale, so that the others lie between codes
    first = torch.zeros(n, dtype=torch.bool, device="cuda")
    first[::BLOCK] = True
    root[first] = 2.0
    (mc, e.ms), (vc, e.vs) = to_8bit(torch.full((n,), 0.5, device="cuda")), to_8bit(root)
    e.m.copy_(mc), e.v.copy_(vc)
    _, r0 = e.moments()
    opt, tl = new_opt(), make_list([e])
    for _ in range(steps):
        opt.step(tl, 1.0, 1.0)
    _, r = e.moments()
    ratio = (r[~first] / r0[~first])
    want = 0.999 ** (steps / 2)
    # each step rounds by at most an eighth of the value (an e4m3 step), with mean 0 and a variance of at most a quarter of
    # the step's square times the share that it moved; 6 standard deviations of the mean over all elements
    deviation = math.sqrt(steps) * 0.125 / 2 / math.sqrt(ratio.numel())
    assert abs(ratio.mean().item() - want) <= 6 * deviation + 1e-4, (ratio.mean().item(), want)


def test_moments_that_are_not_finite():
    torch.manual_seed(8)
    e = Entry(1024)
    e.g[300] = math.nan
    opt = new_opt()
    opt.step(make_list([e]), 1.0, 1.0)
    assert opt.get_norm()[2] == 1
    assert torch.isnan(from_8bit(e.m, e.ms)).all()  # the norm is NaN, so every update is
    # a moment that overflows takes its block with it, and no other
    e = Entry(1024)
    (m, e.ms), (v, e.vs) = zeros_8bit(e.p), zeros_8bit(e.p)
    e.m.copy_(m), e.v.copy_(v)
    e.ms[1], e.vs[1] = math.inf, math.inf
    e.m.view(torch.uint8)[256] = 8
    e.v.view(torch.uint8)[256] = 8
    opt = new_opt()
    opt.step(make_list([e]), 1.0, 1.0)
    values = from_8bit(e.m, e.ms)
    assert not torch.isfinite(values[256:512]).any() and torch.isfinite(values[:256]).all()
    assert torch.isfinite(values[512:]).all() and torch.isfinite(e.p[512:]).all()


def test_tiny_and_huge_values():
    torch.manual_seed(9)
    for std in (1e-12, 1e-30, 1e12):
        e = Entry(2000, std=std)
        (m, e.ms), (v, e.vs) = zeros_8bit(e.p), zeros_8bit(e.p)
        e.m.copy_(m), e.v.copy_(v)
        opt = new_opt()
        opt.step(make_list([e]), 1.0, 1e30)
        m1, r1 = e.moments()
        x = e.g.double()
        if std == 1e-30:  # squares underflow; m is below 2^-100: both are 0
            assert not m1.any() and not r1.any()
            continue
        assert ((m1 - 0.1 * x).abs() <= 0.126 * (0.1 * x).abs() + 0.1 * x.abs().max() / 448 / 512 * 1.01).all()
        assert ((r1 > 0) == (x != 0)).all()


def test_past_2_to_the_32_elements():
    """The last elements of a tensor with more than 2^32."""
    n, tail = (1 << 32) + 700, 1700
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    torch.manual_seed(10)
    small = Entry(tail, torch.bfloat16)
    big = {}
    for name, dtype in (("p", torch.float32), ("g", torch.bfloat16), ("m", torch.uint8), ("v", torch.uint8)):
        big[name] = torch.zeros(n, dtype=dtype, device="cuda")
    at = n - tail
    lead = -at % BLOCK  # the first whole block of the tail
    big["p"][at:], big["g"][at:] = small.p, small.g
    scales = [torch.zeros(-(-n // BLOCK), device="cuda") for _ in range(2)]
    e = Entry(1)
    e.n, e.p, e.g = n, big["p"], big["g"]
    e.m, e.v, (e.ms, e.vs) = big["m"].view(F8), big["v"].view(F8), scales
    opt = new_opt()
    opt.step(make_list([e]), 1.0, 1e30)
    x = small.g.double()[lead:]
    index = torch.arange(at + lead, n, device="cuda")
    bits = chance(index, 1)
    m, r = 0.1 * x, (0.001 * x * x).sqrt()
    block = (at + lead) // BLOCK
    check_codes(e.m[at + lead:], e.ms[block:], m, 8 * U32 * m.abs(), bits & 0xffff, False, "m")
    check_codes(e.v[at + lead:], e.vs[block:], r, 8 * U32 * r, bits >> 16, True, "v")
    assert not e.m.view(torch.uint8)[:1 << 20].any() and not e.ms[:4096].any()


def test_streams():
    torch.manual_seed(11)
    entries = [Entry(100000, torch.bfloat16)]
    start = clones(entries)
    opt, tl = new_opt(), make_list(entries)
    opt.step(tl, 1.0, 1.0)
    want = clones(entries)
    put_back(entries, start)
    torch.cuda.synchronize()
    opt, side = new_opt(), torch.cuda.Stream()
    opt.step(tl, 1.0, 1.0, stream=side)
    side.synchronize()
    assert same(want, clones(entries))


def test_conversion():
    torch.manual_seed(12)
    x = torch.randn(3, 1000, device="cuda")
    codes, scales = to_8bit(x)
    assert codes.shape == x.shape and codes.dtype == F8 and scales.numel() == 12
    back = from_8bit(codes, scales)
    assert ((back - x).abs() <= x.abs() * 2.0 ** -4 * (1 + 2.0 ** -20) + x.abs().max() / 448 * 2.0 ** -10).all()
    codes, scales = zeros_8bit(x)
    assert not from_8bit(codes, scales).any()


def test_a_step_after_a_conversion_stays_bounded():
    """An element whose second moment is far below its block's largest, converted from fp32, then a step without gradient."""
    n = 3 * BLOCK
    m, root = torch.full((n,), 1e-6, device="cuda"), torch.full((n,), 1e-6, device="cuda")
    m[::BLOCK], root[::BLOCK] = 0.01, 1.0
    e = Entry(n)
    e.g.zero_()
    e.p.zero_()
    (mc, e.ms), (vc, e.vs) = to_8bit(m), to_8bit(root, second_moment=True)
    e.m.copy_(mc), e.v.copy_(vc)
    opt = new_opt(step=999, lr=1.0, eps=1e-8)
    opt.step(make_list([e]), 1.0, 1.0)
    bc1, bc2 = 1 - 0.9 ** 1000, 1 - 0.999 ** 1000
    exact = 0.9 * m.double() / bc1 / (math.sqrt(0.999 / bc2) * root.double() + 1e-8)
    # e4m3: m is within 2^-4 of itself and half of the first code, 2^-10 of 1 / 448 of the block's largest; sqrt(v) is not
    # below 1 - 2^-4 of itself (2 % for the step's own fp32 and the parts that these bounds multiply)
    most = exact * (1 + 2.0 ** -4 + 0.01 / 448 * 2.0 ** -10 / m.double()) / (1 - 2.0 ** -4) * 1.02
    assert (-e.p.double() <= most).all() and (e.p <= 0).all()


@pytest.mark.parametrize("eps", [1e-38, 1e-40, 3e-45])
def test_an_eps_that_is_subnormal(eps):
    """Weights without gradient and moments are divided by eps alone: they only decay, as beside fp32 moments."""
    torch.manual_seed(13)
    entries = [Entry(n, grad, shift=shift, eight=eight) for n, grad, shift, eight in (
        (1000, torch.float32, 0, True), (1000, torch.bfloat16, 5, True), (1000, torch.float32, 0, False))]
    for e in entries:
        quiet = torch.rand(e.n, device="cuda") < 0.3
        quiet[256:512] = True
        e.quiet = quiet
        e.g[quiet] = 0
        for t in (e.m, e.v):
            t.view(torch.uint8 if e.eight else torch.float32)[quiet] = 0
        e.guards = [raw.clone() for raw, _ in e.buffers]
    hp = {**HP, "eps": eps}
    want = reference_step(entries, 10, hp, 1.0, 1.0)
    before = [e.p.clone() for e in entries]
    opt = new_opt(step=9, eps=eps)
    opt.step(make_list(entries), 1.0, 1.0)
    check_step(entries, 10, want[2])
    for e, p in zip(entries, before):
        assert torch.isfinite(e.p).all()
        decayed = p[e.quiet].double() * (1 - hp["lr"] * hp["weight_decay"])
        assert ((e.p[e.quiet].double() - decayed).abs() <= 2 * U32 * decayed.abs()).all()


def test_rounding_by_chance_follows_what_moves_against_its_block():
    """One element of each block keeps its moments, and the block its scales, while the others' decay: 0.05 % a step of
    sqrt(v), which rounded to nearest would stay where it is."""
    torch.manual_seed(15)
    n, largest = 1 << 18, 2.0
    e = Entry(n)
    first = torch.zeros(n, dtype=torch.bool, device="cuda")
    first[::BLOCK] = True
    e.g.copy_(torch.where(first, largest, 0.0))  # m and v of constant gradients: the gradient, and its square
    start = torch.where(first, largest, torch.rand(n, device="cuda") * 0.75 + 0.25)
    for codes, scales, second in ((e.m, "ms", False), (e.v, "vs", True)):
        c, s = to_8bit(start, second_moment=second)
        codes.copy_(c)
        setattr(e, scales, s)
    m0, r0 = e.moments()
    # (the test says something: to nearest, one step changes no second moment's code)
    nearest, _ = to_8bit(torch.where(first, r0, r0 * math.sqrt(0.999)).float(), second_moment=True)
    assert torch.equal(nearest.view(torch.uint8), e.v.view(torch.uint8))
    opt, tl = new_opt(), make_list([e])
    # a step of e4m3 is at most an eighth of the value.  A rounding that moves a share f of a step has the variance
    # f (1 - f) steps^2: f is at most 0.0005 x 16 for sqrt(v), whose steps are then 1 / 16 of it (f / 256 = 0.0005 / 16, and
    # 0.0005 / 8 at the other end), and at most 1 / 4 is f (1 - f) for m.  6 deviations of the mean of n elements; 2^-17 of a
    # step is what 16 random bits leave of the mean.
    for steps, left, variance, moments in ((10, 0.9 ** 10, 10 * 0.25 / 64, 0), (400, 0.999 ** 200, 400 * 0.0005 / 8, 1)):
        while opt.get_group_step(0) < steps:
            opt.step(tl, 1.0, 1e30)
        now, before = e.moments()[moments][~first], (m0, r0)[moments][~first]
        ratio = (now / before).mean().item()
        bound = 6 * left * math.sqrt(variance / now.numel()) * 1.1 + left * steps * (2.0 ** -17 / 8 + 8 * U32)
        assert abs(ratio - left) <= bound, (moments, ratio, left, bound)
        assert bound < (1 - left) / 50
        kept = e.moments()[moments][first]
        assert ((kept - largest).abs() <= largest * steps * 8 * U32).all()
