"""What the training operators are measured on: layer norm, linear layer and distillation loss.

`listed()` names the cases, `draw(rng)` makes more of the same ranges, `prepare(case, seed)` makes a case's inputs on the
GPU, `run(state)` makes one pass and `exact(case, seed)` computes the same in 64 bits.  With `own` set, `run` calls
tensor_grad_clip_gb300.ops; otherwise it computes the plain form: elementary torch operations in fp32, rounded once to the
output's type.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
COUNTED = 0.85  # share of the distillation rows that count; the logits of the others need not be read


def listed():
    return [
        # One token of a 4096-wide block: the call's latency.
        dict(name="norm fwd, one token", op="norm_fwd", rows=1, cols=4096, pad=0, dtype="bf16", wdtype="bf16"),
        # The activations of a 16 Ki-token batch entering a block of the 7B list.
        dict(name="norm fwd, 16k tokens", op="norm_fwd", rows=16384, cols=4096, pad=0, dtype="bf16", wdtype="f32"),
        # A block of the 1024-wide action expert trained in fp32.
        dict(name="norm bwd, action expert f32", op="norm_bwd", rows=2500, cols=1024, pad=0, dtype="f32", wdtype="f32"),
        # A long batch of an odd width, its rows inside a wider buffer (a slice of a joint projection's output).
        dict(name="norm bwd, odd width", op="norm_bwd", rows=16381, cols=4099, pad=13, dtype="f16", wdtype="f16"),
        # The 7B list's widest projection for a single token: the weight is read once.
        dict(name="linear fwd, one token", op="linear_fwd", rows=1, n=11008, k=4096, pad=0, dtype="bf16",
             act="silu", residual=False, save=False),
        # The action expert's up projection in training: the backward pass needs the pre-activation too.
        dict(name="linear fwd, expert up", op="linear_fwd", rows=4096, n=4096, k=1024, pad=0, dtype="bf16",
             act="gelu", residual=False, save=True),
        # The 7B list's down projection over a long batch, added to the residual stream.
        dict(name="linear fwd, 16k tokens", op="linear_fwd", rows=16384, n=4096, k=11008, pad=0, dtype="bf16",
             act="none", residual=True, save=False),
        # All three gradients of the action expert's up projection under fp16 training.
        dict(name="linear bwd, expert up", op="linear_bwd", rows=4096, n=4096, k=1024, pad=0, dtype="f16", act="gelu"),
        # The same for a ragged batch and odd widths, where no row starts on a 16-byte boundary.
        dict(name="linear bwd, odd sizes", op="linear_bwd", rows=1021, n=1111, k=1003, pad=0, dtype="bf16", act="silu"),
        # Evaluating a student on a few positions.
        dict(name="distill fwd, few rows", op="distill_fwd", rows=16, vocab=32000, top=32, pad=0, dtype="f32",
             tdtype="f32", masked=0, temperature=1.0),
        # The gradient for a micro-batch whose vocabulary has an odd size.
        dict(name="distill bwd, odd vocabulary", op="distill_bwd", rows=2048, vocab=50021, top=64, pad=0, dtype="bf16",
             tdtype="f32", masked=0, temperature=2.0),
        # A training micro-batch on a large vocabulary padded with masked columns: loss and gradient in one call.
        dict(name="distill loss+grad, 8k rows", op="distill_loss_grad", rows=8192, vocab=131072, top=128, pad=0,
             dtype="bf16", tdtype="bf16", masked=61, temperature=1.5),
    ]


def _between(rng, low, high):
    """A whole number, spread over the logarithm of [low, high]."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _width(rng, low, high):
    """As _between; half of them rounded to a multiple of 64, the other half as they fall."""
    n = _between(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd", "distill_fwd", "distill_bwd",
                     "distill_loss_grad"])
    pad = rng.choice([0, 0, 0, 1, 8, 40])
    if op.startswith("norm"):
        dtype = rng.choice(["f32", "bf16", "f16"])
        cols = _width(rng, 64, 16384)
        return dict(op=op, rows=_between(rng, 1, min(32768, (1 << 26) // cols)), cols=cols, pad=pad, dtype=dtype,
                    wdtype=rng.choice(["f32", dtype]))
    if op.startswith("linear"):
        n, k = _width(rng, 64, 11008), _width(rng, 64, 11008)
        case = dict(op=op, rows=_between(rng, 1, min(16384, (1 << 38) // (n * k))), n=n, k=k, pad=pad,
                    dtype=rng.choice(["bf16", "f16"]), act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
        return dict(case, residual=rng.random() < 0.5, save=rng.random() < 0.5) if op == "linear_fwd" else case
    vocab = _width(rng, 1000, 262144)
    return dict(op=op, rows=_between(rng, 1, min(16384, (1 << 29) // vocab)), vocab=vocab,
                top=_between(rng, 1, 256), pad=pad, dtype=rng.choice(["f32", "bf16", "f16"]),
                tdtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0, 0, 5, 61]),
                temperature=rng.choice([1.0, 1.5, 2.0, 4.0]))


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"].startswith("norm"):
        r, c, we = case["rows"], case["cols"], SIZES[case["wdtype"]]
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * r * c * e + 2 * c * we + 8 * r, "flops": 8 * r * c}
        return {"bytes": 3 * r * c * e + 3 * c * we + 8 * r, "flops": 14 * r * c}
    if case["op"].startswith("linear"):
        m, n, k = case["rows"], case["n"], case["k"]
        if case["op"] == "linear_fwd":
            outs = 1 + int(case["residual"]) + int(case["save"])
            return {"bytes": (m * k + n * k + n + outs * m * n) * e, "flops": 2 * m * n * k}
        reads = 1 if case["act"] == "none" else 2
        return {"bytes": (reads * m * n + 2 * m * k + 2 * n * k + n) * e, "flops": 4 * m * n * k}
    r, v, t = case["rows"], case["vocab"], case["top"]
    counted = COUNTED * (r - 1) + 1
    small = counted * t * (4 + SIZES[case["tdtype"]]) + 8 * r
    if case["op"] == "distill_fwd":
        return {"bytes": counted * v * e + small, "flops": 5 * counted * v}
    return {"bytes": (counted + r) * v * e + small, "flops": 9 * counted * v}


def _rows(gen, rows, cols, pad, dtype, std=1.0):
    """[rows, cols] of N(0, std); with `pad`, a slice of a buffer whose rows are that much longer."""
    buf = torch.empty(rows, cols + pad, device="cuda", dtype=dtype)
    for at in range(0, rows, 2048):  # drawn in fp32 a few rows at a time
        n = min(2048, rows - at)
        buf[at:at + n] = torch.randn(n, cols + pad, device="cuda", generator=gen) * std
    return buf[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]

    def vector(n, dtype, mean, std):
        return (torch.randn(n, device="cuda", generator=gen) * std + mean).to(dtype)

    if case["op"].startswith("norm"):
        r, c, wdt = case["rows"], case["cols"], DTYPES[case["wdtype"]]
        s["x"] = _rows(gen, r, c, case["pad"], dt)
        # rows of a residual stream: a scale and an offset of their own, and a few channels far larger than the rest
        s["x"].mul_(vector(r, dt, 1.5, 0.3)[:, None]).add_(vector(r, dt, 0.25, 0.5)[:, None])
        s["x"][:, :: max(1, c // 3)].mul_(8.0)
        s["weight"], s["bias"] = vector(c, wdt, 1.0, 0.2), vector(c, wdt, 0.0, 0.2)
        if case["op"] == "norm_bwd":
            s["dy"] = _rows(gen, r, c, case["pad"], dt, 1e-2)
            s["mean"], s["rstd"] = torch.empty(r, device="cuda"), torch.empty(r, device="cuda")
            for at in range(0, r, 2048):
                x = s["x"][at:at + 2048].double()
                var, mean = torch.var_mean(x, dim=1, unbiased=False)
                s["mean"][at:at + 2048], s["rstd"][at:at + 2048] = mean, 1.0 / torch.sqrt(var + EPS)
    elif case["op"].startswith("linear"):
        m, n, k = case["rows"], case["n"], case["k"]
        s["x"] = _rows(gen, m, k, case["pad"], dt)
        s["weight"] = _rows(gen, n, k, case["pad"], dt, 1.0 / math.sqrt(k))
        if case["op"] == "linear_fwd":
            s["bias"] = vector(n, dt, 0.0, 0.1)
            s["res"] = _rows(gen, m, n, case["pad"], dt) if case["residual"] else None
        else:
            s["dy"] = _rows(gen, m, n, case["pad"], dt, 1e-2)
            s["z"] = None if case["act"] == "none" else _rows(gen, m, n, case["pad"], dt)
    else:
        r, v, t = case["rows"], case["vocab"], case["top"]
        z = _rows(gen, r, v, case["pad"], dt, 2.5)
        if case["masked"]:
            z[:, v - case["masked"]:] = -math.inf  # padding of the vocabulary: never predicted
        # one entry out of each of `top` equal parts of the real vocabulary, likelier to the teacher than the rest
        part = (v - case["masked"]) // t
        index = torch.arange(t, device="cuda") * part + torch.randint(0, part, (r, t), device="cuda", generator=gen)
        logit = z.gather(1, index).float() * 0.7 + torch.randn(r, t, device="cuda", generator=gen) + 4.0
        logit, order = logit.sort(dim=1, descending=True)
        index = index.gather(1, order)
        # some teachers answer with fewer entries: the rest is marked with -1
        short = torch.rand(r, 1, device="cuda", generator=gen) < 0.1
        index[short & (torch.arange(t, device="cuda") >= (t + 1) // 2)] = -1
        s["logits"], s["teacher"], s["index"] = z, logit.to(DTYPES[case["tdtype"]]), index.int()
        # prompt and padding positions do not count; the others are averaged
        keep = (torch.rand(r, device="cuda", generator=gen) < COUNTED).float()
        keep[0] = 1.0
        s["row_weight"] = keep / max(1, r)
        if case["op"] == "distill_bwd":
            s["grad_loss"] = vector(r, torch.float32, 1.0, 0.1)
            s["lse"] = torch.empty(r, device="cuda")
            for at in range(0, r, 512):
                s["lse"][at:at + 512] = torch.logsumexp(z[at:at + 512].double() / case["temperature"], dim=1)
    return s


def run(state):
    return (_own if own else _plain)[state["op"]](state)


# ---- the framework's operators -------------------------------------------


def _own_norm_fwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS)


def _own_norm_bwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])


def _own_linear_fwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.linear_forward(s["x"], s["weight"], s["bias"], activation=s["act"], residual=s["res"],
                              save_preactivation=s["save"])


def _own_linear_bwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.linear_backward(s["dy"], s["x"], s["weight"], s["z"], activation=s["act"])


def _own_distill_fwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.distill_forward(s["logits"], s["teacher"], s["index"], temperature=s["temperature"],
                               row_weight=s["row_weight"])


def _own_distill_bwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.distill_backward(s["grad_loss"], s["logits"], s["lse"], s["teacher"], s["index"],
                                temperature=s["temperature"], row_weight=s["row_weight"])


def _own_distill_loss_grad(s):
    from tensor_grad_clip_gb300 import ops
    return ops.distill_loss_grad(s["logits"], s["teacher"], s["index"], temperature=s["temperature"],
                                 row_weight=s["row_weight"])


_own = dict(norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd, linear_fwd=_own_linear_fwd, linear_bwd=_own_linear_bwd,
            distill_fwd=_own_distill_fwd, distill_bwd=_own_distill_bwd, distill_loss_grad=_own_distill_loss_grad)


# ---- their plain forms ----------------------------------------------------


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(dim=1)
    d = x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(dim=1) + EPS)
    y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"].float()
    dx = (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
    return dx.to(s["x"].dtype), (dy * xh).sum(dim=0).to(s["weight"].dtype), dy.sum(dim=0).to(s["weight"].dtype)


def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _plain_linear_fwd(s):
    z = s["x"].float() @ s["weight"].float().t() + s["bias"].float()
    y = _act(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    dt = s["x"].dtype
    return (y.to(dt), z.to(dt)) if s["save"] else y.to(dt)


def _plain_linear_bwd(s):
    dz, dt = s["dy"].float(), s["x"].dtype
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    return (dz @ s["weight"].float()).to(dt), (dz.t() @ s["x"].float()).to(dt), dz.sum(dim=0).to(dt)


def _teacher(s):
    """p, log p of the valid entries (p = 0 elsewhere) and the entries' places."""
    valid = (s["index"] >= 0) & (s["index"] < s["vocab"])
    t = torch.where(valid, s["teacher"].float() / s["temperature"], -math.inf)
    top = t.max(dim=1, keepdim=True).values
    top = torch.where(top == -math.inf, 0.0, top)
    total = torch.exp(t - top).sum(dim=1, keepdim=True)
    logp = t - top - torch.log(total)
    p = torch.where(total > 0, torch.exp(logp), 0.0)
    return p, logp, torch.where(valid, s["index"], 0).long()


def _plain_lse(s):
    z = s["logits"].float() / s["temperature"]
    top = z.max(dim=1, keepdim=True).values
    return z, top[:, 0] + torch.log(torch.exp(z - top).sum(dim=1))


def _plain_loss(s, z, lse):
    p, logp, at = _teacher(s)
    each = torch.where(p > 0, p * (logp - z.gather(1, at) + lse[:, None]), 0.0)
    w = s["row_weight"]
    return torch.where(w != 0, w * s["temperature"] ** 2 * each.sum(dim=1), 0.0)


def _plain_gradient(s, z, lse, scale):
    p, _, at = _teacher(s)
    dz = torch.exp(z - lse[:, None]) * (p.sum(dim=1, keepdim=True) > 0)
    dz.scatter_add_(1, at, -p)
    dz = torch.where((scale != 0)[:, None], dz * (scale * s["temperature"])[:, None], 0.0)
    return dz.to(s["logits"].dtype)


def _plain_distill_fwd(s):
    z, lse = _plain_lse(s)
    return _plain_loss(s, z, lse), torch.where(s["row_weight"] != 0, lse, 0.0)


def _plain_distill_bwd(s):
    z = s["logits"].float() / s["temperature"]
    return _plain_gradient(s, z, s["lse"], s["grad_loss"] * s["row_weight"])


def _plain_distill_loss_grad(s):
    z, lse = _plain_lse(s)
    return _plain_loss(s, z, lse), _plain_gradient(s, z, lse, s["row_weight"])


_plain = dict(norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd, linear_fwd=_plain_linear_fwd,
              linear_bwd=_plain_linear_bwd, distill_fwd=_plain_distill_fwd, distill_bwd=_plain_distill_bwd,
              distill_loss_grad=_plain_distill_loss_grad)


# ---- the definitions in 64 bits ---------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm_fwd":
        x = s["x"].double()
        mean = x.sum(1) / case["cols"]
        second = ((x - mean.unsqueeze(1)) ** 2).sum(1) / case["cols"]
        rstd = (second + EPS) ** -0.5
        return (x - mean.unsqueeze(1)).mul_(rstd.unsqueeze(1)) * s["weight"].double() + s["bias"].double(), mean, rstd
    if case["op"] == "norm_bwd":
        n = case["cols"]
        dy, rstd = s["dy"].double(), s["rstd"].double().unsqueeze(1)
        xh = (s["x"].double() - s["mean"].double().unsqueeze(1)) * rstd
        g = dy * s["weight"].double()
        along = torch.einsum("rc,rc->r", g, xh).unsqueeze(1) / n
        dx = rstd * (g - g.sum(1, keepdim=True) / n - xh * along)
        return dx, torch.einsum("rc,rc->c", dy, xh), dy.sum(0)
    if case["op"].startswith("linear"):
        act = case["act"]
        normal = torch.distributions.Normal(torch.zeros((), device="cuda", dtype=torch.float64), 1.0)
        if case["op"] == "linear_fwd":
            z = torch.addmm(s["bias"].double(), s["x"].double(), s["weight"].double().t())
        else:
            z = s["z"].double() if s["z"] is not None else None
        if act in ("gelu_tanh", "silu") and z is not None:
            # 0.5 (1 + tanh u) is the logistic function of 2u
            u = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            gate = torch.sigmoid(u)
        if case["op"] == "linear_fwd":
            y = {"none": lambda: z.clone(), "relu": lambda: z.clamp(min=0), "gelu": lambda: z * normal.cdf(z)}.get(
                act, lambda: z * gate)()
            if s["res"] is not None:
                y += s["res"].double()
            return (y, z) if case["save"] else y
        dz = s["dy"].double()
        if act == "relu":
            dz = dz * (z > 0)
        elif act == "gelu":
            dz = dz * (normal.cdf(z) + z * torch.exp(normal.log_prob(z)))
        elif act == "silu":
            dz = dz * (gate + z * gate * (1 - gate))
        elif act == "gelu_tanh":
            dz = dz * (gate + z * gate * (1 - gate) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2))
        return dz @ s["weight"].double(), dz.t() @ s["x"].double(), dz.sum(0)
    # distillation, a few hundred rows at a time
    temp, v = case["temperature"], case["vocab"]
    losses, lses, grads = [], [], []
    for at in range(0, case["rows"], 256):
        part = slice(at, at + 256)
        z = s["logits"][part].double() / temp
        lse = s["lse"][part].double() if case["op"] == "distill_bwd" else torch.logsumexp(z, 1)
        index = s["index"][part].long()
        t = (s["teacher"][part].double() / temp).masked_fill((index < 0) | (index >= v), -math.inf)
        p = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)  # no valid entry at all: no teacher
        index = index.clamp(0, v - 1)
        w = s["row_weight"][part].double()
        if case["op"] != "distill_bwd":
            # cross entropy less the teacher's entropy
            logq = z.gather(1, index) - lse.unsqueeze(1)
            cross = -(p * logq).masked_fill(p == 0, 0.0).sum(1)
            losses.append((w * temp * temp * (cross + torch.xlogy(p, p).sum(1))).masked_fill(w == 0, 0.0))
            lses.append(lse.masked_fill(w == 0, 0.0))
        if case["op"] != "distill_fwd":
            if case["op"] == "distill_bwd":
                w = w * s["grad_loss"][part].double()
            d = torch.exp(z - lse.unsqueeze(1)) * p.sum(1, keepdim=True)
            d.scatter_add_(1, index, -p)
            grads.append((d * (w * temp).unsqueeze(1)).masked_fill((w == 0).unsqueeze(1), 0.0))
    if case["op"] == "distill_fwd":
        return torch.cat(losses), torch.cat(lses)
    if case["op"] == "distill_bwd":
        return torch.cat(grads)
    return torch.cat(losses), torch.cat(grads)
