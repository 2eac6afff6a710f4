"""The training operators' formulas in fp64 (torch, any device), written from
their definitions, and error bounds of an fp32 computation of them.

A bound has two parts: half a unit in the last place of the output's type
(one rounding), and fp32 arithmetic: a sum of n terms in any order errs by at
most n * 2^-24 times the sum of the terms' magnitudes; the few other
operations add a small constant number of such units."""
import math

import torch

U32 = 2.0 ** -24
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}  # underflow


def rounding(ref, dtype):
    return HALF_ULP[dtype] * ref.abs() + TINY[dtype]


def assert_close(got, ref, tol, what=""):
    """|got - ref| <= tol where ref is finite; the same infinities and NaN elsewhere."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN elsewhere than expected"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    over = ((got - ref).abs() > tol) & fine
    if over.any():
        k = int(((got - ref).abs() / tol.expand_as(ref).clamp(min=1e-300)).masked_fill(~fine, 0).argmax())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} off; worst at {k}: "
                             f"{got.flatten()[k].item()} for {ref.flatten()[k].item()}, "
                             f"bound {tol.expand_as(ref).flatten()[k].item()}")


# ---- layer norm -------------------------------------------------------------

def norm_stats(x, eps):
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    return mean, 1 / torch.sqrt(var + eps)


def norm_forward(x, w, b, eps):
    mean, rstd = norm_stats(x, eps)
    y = (x.double() - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


def _units(n):
    # partial sums run over at most 256 terms in sequence before a tree joins them
    return (min(n, 256) + 32) * U32


def norm_forward_bounds(x, w, b, eps, y, mean, rstd):
    u = _units(x.shape[1])
    x = x.double()
    size = x.abs().mean(1)                          # magnitude that the mean's sum sees
    tol_mean = u * size + rounding(mean, torch.float32)
    # The variance is a sum of squares of d = x - mean: d errs by tol_mean and one
    # rounding, which moves the variance by at most 2 std * tol + tol^2.
    std = torch.sqrt((1 / rstd ** 2 - eps).clamp(min=0))
    e = tol_mean + U32 * (size + mean.abs())
    dvar = u / rstd ** 2 + 2 * std * e + e * e
    rel = 0.5 * dvar * rstd ** 2 * (1 + dvar * rstd ** 2) + 4 * U32
    tol_rstd = rstd * rel
    wa = 1.0 if w is None else w.double().abs()
    ba = 0.0 if b is None else b.double().abs()
    xh = (x - mean[:, None]).abs() * rstd[:, None]
    # the last four roundings, on the product and on the sum with the bias
    tol = wa * (e[:, None] * rstd[:, None] * (1 + rel[:, None]) + xh * rel[:, None]) + 8 * U32 * (wa * xh + ba)
    return tol, tol_mean, tol_rstd


def norm_backward(dy, x, w, mean, rstd):
    dy, x = dy.double(), x.double()
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy if w is None else dy * w.double()
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def norm_backward_bounds(dy, x, w, mean, rstd):
    u = _units(x.shape[1])
    dy, x, mean, rstd = dy.double().abs(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    g = dy if w is None else dy * w.double().abs()
    xa = rstd * (x.abs() + mean.abs())  # |xh| and the magnitude its rounding errors go with
    dx = u * rstd * (g + g.mean(1, keepdim=True) + xa * (g * xa).mean(1, keepdim=True) * 2)
    n = (x.shape[0] + 16) * U32
    return dx, n * (dy * xa).sum(0), n * dy.sum(0)


# ---- linear layer -------------------------------------------------------------

def activate(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def linear_forward(x, w, b, act, res):
    z = x.double() @ w.double().t()
    if b is not None:
        z = z + b.double()
    y = activate(z, act)
    return (y if res is None else y + res.double()), z


def _product_units(k):
    # a tensor core may drop, rather than round, the last bit of each partial sum
    return (k + 8) * 2 * U32


def linear_forward_bounds(x, w, b, act, res):
    size = x.double().abs() @ w.double().abs().t()
    if b is not None:
        size = size + b.double().abs()
    tol_z = _product_units(x.shape[1]) * size
    # every activation's slope is at most 1.13 in magnitude; 16 units of its value for its own evaluation
    tol_y = 1.13 * tol_z + 16 * U32 * (size + (0 if res is None else res.double().abs()))
    return tol_y, tol_z


def linear_backward(dy, x, w, z, act):
    dz = dy.double() if act == "none" else dy.double() * act_slope(z.double(), act)
    return dz @ w.double(), dz.t() @ x.double(), dz.sum(0)


def linear_backward_bounds(dy, x, w, z, act, dtype):
    dza = dy.double().abs() * (1.0 if act == "none" else act_slope(z.double(), act).abs())
    # the slope's own evaluation, and with an activation the rounding of dz to 16 bits
    err = 16 * U32 * 1.2 * dy.double().abs() if act != "none" else torch.zeros_like(dza)
    err16 = err + (rounding(dza, dtype) if act != "none" else 0)
    wa, xa = w.double().abs(), x.double().abs()
    dx = _product_units(w.shape[0]) * (dza @ wa) + err16 @ wa
    dw = _product_units(x.shape[0]) * (dza.t() @ xa) + err16.t() @ xa
    db = (x.shape[0] + 16) * U32 * dza.sum(0) + err.sum(0)
    return dx, dw, db


# ---- distillation loss ----------------------------------------------------------

def distill_parts(logits, teacher, index, T):
    """log q, lse, p, log p (0 where p is 0), clipped index."""
    z = logits.double() / T
    lse = torch.logsumexp(z, 1)
    vocab = logits.shape[1]
    ok = (index >= 0) & (index < vocab)
    t = torch.where(ok, teacher.double() / T, -math.inf)
    if t.shape[1] == 0:
        p = t
    else:
        p = torch.softmax(t, 1)
        p = torch.where((t == -math.inf).all(1, keepdim=True), torch.zeros_like(p), p)
    return z, lse, t, p, torch.where(ok, index.long(), torch.zeros_like(index.long()))


def distill(logits, teacher, index, T, weight=None, grad_loss=None, lse=None):
    """loss, lse, dlogits (of sum(loss * grad_loss)), in fp64."""
    z, own, t, p, at = distill_parts(logits, teacher, index, T)
    lse = own if lse is None else lse.double()
    w = torch.ones_like(lse) if weight is None else weight.double()
    g = w if grad_loss is None else w * grad_loss.double()
    each = torch.xlogy(p, p) - torch.where(p > 0, p * (z.gather(1, at) - lse[:, None]), torch.zeros_like(p))
    loss = torch.where(w != 0, w * T * T * each.sum(1), torch.zeros_like(w))
    q = torch.exp(z - lse[:, None])
    any_ = (p > 0).any(1, keepdim=True) | torch.isnan(p).any(1, keepdim=True)
    d = torch.where(any_, q, torch.zeros_like(q))
    d = d.scatter_add(1, at, -p) * (g * T)[:, None]
    d = torch.where((g != 0)[:, None] & any_, d, torch.zeros_like(d))
    return loss, torch.where(w != 0, lse, torch.zeros_like(lse)), d


def distill_bounds(logits, teacher, index, T, weight=None, grad_loss=None):
    z, lse, t, p, at = distill_parts(logits, teacher, index, T)
    c = 64 * U32  # exponentials within a few units, sums over at most about 50 terms in sequence per thread
    big = lambda a: torch.nan_to_num(a, nan=0.0, posinf=0.0, neginf=0.0).abs()  # noqa: E731
    w = torch.ones_like(lse) if weight is None else weight.double()
    g = w if grad_loss is None else w * grad_loss.double()
    zj = z.gather(1, at)
    reach = 1 + big(t) + big(t).amax(1, keepdim=True) if t.shape[1] else 1 + big(t)
    top = big(z).masked_fill(torch.isinf(z), 0).amax(1)
    tol_lse = c * (1 + big(lse) + torch.where(torch.isfinite(lse), big(z.amax(1)), torch.zeros_like(lse)))
    diff = big(torch.log(p.clamp(min=1e-300)) - zj + lse[:, None])
    tol_loss = w.abs() * T * T * c * (p * (reach + big(zj) + big(lse)[:, None]) * (1 + diff)).sum(1) + \
        w.abs() * T * T * tol_lse * p.sum(1)
    q = torch.exp(z - lse[:, None])
    tol_d = c * torch.nan_to_num(q) * (1 + big(z) + big(lse)[:, None])
    tol_d = tol_d.scatter_add(1, at, c * p * reach.expand_as(p)) * (g.abs() * T)[:, None]
    del top
    return tol_loss + TINY[torch.float32], tol_lse, tol_d
