"""What the operators of a language model's two ends and its optimizer are measured on: embedding lookup with its
gradient by sorted tokens, softmax cross entropy of a linear head over a large vocabulary without its logits in memory,
and the clipped AdamW step with moments held in 8 bits.

`listed()` names the cases, `draw(rng)` makes more of the same ranges, `prepare(case, seed)` makes a case's inputs on the
GPU, `run(state)` makes one pass and `exact(case, seed)` computes the same in 64 bits.  With `own` set, `run` calls
tensor_grad_clip_gb300; otherwise it computes the plain form: elementary torch operations in fp32 (64 bits for the sum of
squares of all gradients), rounded once to the output's type.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
COUNTED = 0.85   # share of the rows that count in the loss
PADDING = 0.03   # share of the positions that hold no token

# The optimizer's settings: AdamW on every list.
LR, BETA1, BETA2, EPS, DECAY = 5e-6, 0.9, 0.999, 1e-8, 0.01
DIVISOR, MAX_NORM = 64.0, 1.0
BLOCK = 256      # elements that share a scale
TOP = 448.0      # the largest 8-bit value (e4m3)


def listed():
    return [
        # Looking one token up in a generation loop: the call's latency.
        dict(name="embedding one token", op="emb_fwd", rows=1, vocab=32000, cols=4096, pad=0, dtype="bf16", index="i64",
             scale=1.0),
        # The tokens of a training batch, scaled by the square root of the width.
        dict(name="embedding 16k tokens", op="emb_fwd", rows=16384, vocab=131072, cols=4096, pad=0, dtype="bf16",
             index="i64", scale=64.0),
        # The gradient of that table's smaller sister: frequent tokens stand in thousands of places.
        dict(name="embedding grad 16k tokens", op="emb_bwd", rows=16384, vocab=32000, cols=4096, pad=0, dtype="bf16",
             index="i64", scale=1.0, tied=False),
        # A table of odd sizes that the head shares: the gradient is added to the head's.
        dict(name="embedding grad tied odd", op="emb_bwd", rows=5003, vocab=50021, cols=1003, pad=5, dtype="f32",
             index="i32", scale=2.0, tied=True),
        # Scoring a few positions: the head's weight is read once.
        dict(name="head loss few rows", op="head_fwd", rows=16, vocab=32000, k=1024, pad=0, dtype="bf16", index="i64"),
        # The loss of a validation batch.
        dict(name="head loss 8k rows", op="head_fwd", rows=8192, vocab=32000, k=4096, pad=0, dtype="bf16", index="i64"),
        # Both gradients of a ragged batch on a vocabulary and a width of odd sizes.
        dict(name="head grad odd sizes", op="head_bwd", rows=1021, vocab=50021, k=1003, pad=3, dtype="bf16",
             index="i32"),
        # A training micro-batch of the action expert's width in fp16: loss and gradients in one call.
        dict(name="head loss+grad expert f16", op="head_loss_grad", rows=2500, vocab=32000, k=1024, pad=0, dtype="f16",
             index="i64"),
        # A training micro-batch of the 7B list's width on a large vocabulary.
        dict(name="head loss+grad 4k rows", op="head_loss_grad", rows=4096, vocab=131072, k=4096, pad=0, dtype="bf16",
             index="i64"),
        # A few small tensors: the step's latency.
        dict(name="adamw 8 bits small list", op="adamw", count=12, low=16, high=16384, layout=1, whole=0, grad="f32",
             masters=False, step=10, norm=5.0),
        # A list of ragged tensors, a quarter of which keep their moments in 32 bits.
        dict(name="adamw 8 bits ragged list", op="adamw", count=600, low=3, high=600000, layout=2, whole=150, grad="f32",
             masters=False, step=1000, norm=0.5),
        # The 302 M parameters of the action expert: bf16 gradients, bf16 copies of the fp32 weights.
        dict(name="adamw 8 bits 302M", op="adamw", count=72, low=4194304, high=4195840, layout=3, whole=4, grad="bf16",
             masters=True, step=2000, norm=20.0),
    ]


def _between(rng, low, high):
    """A whole number, spread over the logarithm of [low, high]."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _width(rng, low, high):
    """As _between; half of them rounded to a multiple of 64, the other half as they fall."""
    n = _between(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["emb_fwd", "emb_bwd", "head_fwd", "head_bwd", "head_loss_grad", "adamw"])
    pad = rng.choice([0, 0, 0, 1, 8, 40])
    index = rng.choice(["i32", "i64"])
    if op.startswith("emb"):
        cols = _width(rng, 64, 8192)
        vocab = _width(rng, 1000, min(262144, (1 << 29) // cols))
        case = dict(op=op, rows=_between(rng, 1, min(65536, (1 << 26) // cols)), vocab=vocab, cols=cols, pad=pad,
                    dtype=rng.choice(["f32", "bf16", "f16"]), index=index, scale=rng.choice([1.0, 0.5, math.sqrt(cols)]))
        return dict(case, tied=rng.random() < 0.3) if op == "emb_bwd" else case
    if op.startswith("head"):
        k, vocab = _width(rng, 64, 4096), _width(rng, 1000, 131072)
        return dict(op=op, rows=_between(rng, 1, min(8192, (1 << 39) // (k * vocab))), vocab=vocab, k=k, pad=pad,
                    dtype=rng.choice(["bf16", "f16"]), index=index)
    count, low = _between(rng, 1, 600), _between(rng, 1, 4096)
    high = _between(rng, low, max(low, (1 << 27) // count))
    return dict(op=op, count=count, low=low, high=high, layout=rng.randrange(1 << 20), whole=rng.randrange(count // 2 + 1),
                grad=rng.choice(["f32", "bf16", "f16"]), masters=rng.random() < 0.5, step=_between(rng, 1, 10000),
                norm=rng.choice([0.5, 5.0]))


def _sizes(case):
    """(elements of the tensors with moments in 8 bits, of those with moments in 32)."""
    rng = random.Random(case["layout"])
    n = [_between(rng, case["low"], case["high"]) for _ in range(case["count"])]
    return n[case["whole"]:], n[:case["whole"]]


def _distinct(rows, vocab):
    """How many different tokens _tokens draws, on average."""
    n = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = torch.log1p(1 / n) / math.log(vocab)
    return (1 - torch.exp(rows * (1 - PADDING) * torch.log1p(-p.clamp(max=0.5)))).sum().item()


def work(case):
    if case["op"].startswith("emb"):
        r, v, c, e = case["rows"], case["vocab"], case["cols"], SIZES[case["dtype"]]
        index = r * (4 if case["index"] == "i32" else 8)
        if case["op"] == "emb_fwd":
            return {"bytes": (_distinct(r, v) + r) * c * e + index, "flops": r * c}
        # a tied gradient is read and written where there are tokens, another is written whole
        out = 2 * _distinct(r, v) if case["tied"] else v
        return {"bytes": (r + out) * c * e + index, "flops": 2 * r * c}
    if case["op"].startswith("head"):
        v, k, e = case["vocab"], case["k"], SIZES[case["dtype"]]
        r = max(1.0, COUNTED * case["rows"])
        if case["op"] == "head_fwd":
            return {"bytes": (r + v) * k * e + 16 * r, "flops": 2 * r * v * k}
        return {"bytes": 2 * (r + v) * k * e + 16 * r, "flops": 6 * r * v * k}
    small, whole = (sum(n) for n in _sizes(case))
    g, copy = SIZES[case["grad"]], 2 if case["masters"] else 0
    return {"bytes": small * (2 * g + 8 + 4 + 16 / BLOCK + copy) + whole * (2 * g + 24 + copy),
            "flops": 20 * (small + whole)}


def _rows(gen, rows, cols, pad, dtype, std=1.0):
    """[rows, cols] of N(0, std); with `pad`, a slice of a buffer whose rows are that much longer."""
    buf = torch.empty(rows, cols + pad, device="cuda", dtype=dtype)
    for at in range(0, rows, 8192):  # drawn in fp32 a few rows at a time
        n = min(8192, rows - at)
        buf[at:at + n] = torch.randn(n, cols + pad, device="cuda", generator=gen) * std
    return buf[:, :cols]


def _tokens(gen, rows, vocab):
    """Tokens of a text: the n-th most frequent one is 1 / n as likely as the first; their numbers are scattered."""
    rank = torch.exp(torch.rand(rows, device="cuda", generator=gen, dtype=torch.float64) * math.log(vocab)).long() - 1
    return rank.clamp(0, vocab - 1) * 7919 % vocab


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "adamw":
        return _prepare_adamw(s, gen)
    dt, r, v = DTYPES[case["dtype"]], case["rows"], case["vocab"]
    tokens = _tokens(gen, r, v)
    tokens[(torch.rand(r, device="cuda", generator=gen) < PADDING) & (torch.arange(r, device="cuda") > 0)] = -1
    s["index"] = tokens.int() if case["index"] == "i32" else tokens
    if case["op"] == "emb_fwd":
        s["table"] = _rows(gen, v, case["cols"], case["pad"], dt, 0.02)
    elif case["op"] == "emb_bwd":
        s["dy"] = _rows(gen, r, case["cols"], case["pad"], dt, 1e-2)
        s["out"] = _rows(gen, v, case["cols"], 0, dt, 1e-2) if case["tied"] else None
    else:
        k = case["k"]
        s["weight"] = _rows(gen, v, k, case["pad"], dt, 1.0 / math.sqrt(k))
        # a model that has learned something: each row leans towards its token, by a strength of its own (not so far
        # that a loss is near 0, where fp32 leaves it no digits)
        s["x"] = _rows(gen, r, k, case["pad"], dt, 2.0)
        lean = torch.randn(r, 1, device="cuda", generator=gen) * 2.0 + 5.0
        s["x"].add_((s["weight"][tokens.clamp(min=0)].float() * lean).to(dt))
        # prompt positions do not count; the others are averaged, under a loss scale in fp16
        keep = (torch.rand(r, device="cuda", generator=gen) < COUNTED / (1 - PADDING)).float()
        keep[0] = 1.0
        s["row_weight"] = keep / r * (1024.0 if case["dtype"] == "f16" else 1.0)
        if case["op"] == "head_bwd":
            s["grad_loss"] = torch.randn(r, device="cuda", generator=gen) * 0.1 + 1.0
            s["lse"] = torch.empty(r, device="cuda")
            for at in range(0, r, 1024):
                z = s["x"][at:at + 1024].float() @ s["weight"].float().t()
                s["lse"][at:at + 1024] = torch.logsumexp(z.double(), dim=1)
    return s


def _prepare_adamw(s, gen):
    """Flat buffers, each tensor from a multiple of BLOCK elements on, and the tensors as their parts."""
    dt = DTYPES[s["grad"]]
    for part, sizes in zip(("small", "whole"), _sizes(s)):
        blocks = torch.tensor([-(-n // BLOCK) for n in sizes], dtype=torch.int64)
        first = blocks.cumsum(0) - blocks
        total = int(blocks.sum()) * BLOCK
        at = [int(i) * BLOCK for i in first]
        # elements of padding stay 0
        ids = torch.repeat_interleave(torch.arange(len(sizes)), blocks).cuda()
        s[part + ".block"] = torch.arange(total // BLOCK, device="cuda") - first.cuda()[ids]
        left = torch.tensor(sizes, device="cuda", dtype=torch.int64)[ids] - s[part + ".block"] * BLOCK
        real = (torch.arange(BLOCK, device="cuda") < left[:, None]).reshape(-1)

        def normal(std):
            return torch.randn(total, device="cuda", generator=gen).mul_(std).mul_(real)
        p = normal(0.02)
        g = normal(1.0).to(dt)
        # rows of an embedding without a token and other quiet blocks: no gradient
        g.view(-1, BLOCK)[torch.rand(total // BLOCK, device="cuda", generator=gen) < 0.05] = 0
        spread = torch.exp(torch.randn(total // BLOCK, 1, device="cuda", generator=gen))  # each block's own scale
        if part == "small":
            codes = {"m": normal(100.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn),
                     "v": normal(100.0).abs_().clamp_(max=TOP).to(torch.float8_e4m3fn)}
            scales = {"m": spread[:, 0] * 1e-5, "v": spread[:, 0] * 3e-5}
            s.update({"small.m": codes["m"], "small.v": codes["v"], "small.ms": scales["m"], "small.vs": scales["v"]})
            s["ms"] = [scales["m"][int(i):int(i + n)] for i, n in zip(first, blocks)]
            s["vs"] = [scales["v"][int(i):int(i + n)] for i, n in zip(first, blocks)]
        else:
            s["whole.m"] = (normal(1e-3).view(-1, BLOCK) * spread).view(-1)
            s["whole.v"] = (normal(3e-3).view(-1, BLOCK) * spread).view(-1).square_()
        s[part + ".p"], s[part + ".g"] = p, g
        s[part + ".copy"] = p.bfloat16() if s["masters"] else None
        for name in ("p", "g", "m", "v", "copy"):
            flat = s[f"{part}.{name}"]
            s.setdefault(name, []).extend([None if flat is None else flat[a:a + n] for a, n in zip(at, sizes)])
    # gradients of the norm that the case says, before the clipping
    total = math.sqrt(sum(s[f"{part}.g"].double().square().sum().item() for part in ("small", "whole")))
    for part in ("small", "whole"):
        s[part + ".g"].mul_(s["norm"] * DIVISOR / max(total, 1e-30))
    return s


def run(state):
    return (_own if own else _plain)[state["op"]](state)


# ---- the framework's operators -------------------------------------------


def _own_emb_fwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.embedding_forward(s["index"], s["table"], scale=s["scale"])


def _own_emb_bwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.embedding_backward(s["dy"], s["index"], s["vocab"], scale=s["scale"], out=s["out"])


def _own_head_fwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.linear_cross_entropy_forward(s["x"], s["weight"], s["index"], row_weight=s["row_weight"])


def _own_head_bwd(s):
    from tensor_grad_clip_gb300 import ops
    return ops.linear_cross_entropy_backward(s["grad_loss"], s["x"], s["weight"], s["index"], s["lse"],
                                             row_weight=s["row_weight"])


def _own_head_loss_grad(s):
    from tensor_grad_clip_gb300 import ops
    return ops.linear_cross_entropy_loss_grad(s["x"], s["weight"], s["index"], row_weight=s["row_weight"])


def _own_adamw(s):
    from tensor_grad_clip_gb300 import SomaOpt, TensorList
    if "opt" not in s:  # made once, as a program does before its first step
        s["opt"] = opt = SomaOpt(device=torch.cuda.current_device())
        opt.add_group(lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY)
        opt.set_group_step(0, s["step"] - 1)
        n = len(s["p"])
        none = [None] * s["whole"]
        s["list"] = TensorList(s["p"], s["g"], s["m"], s["v"], groups=[0] * n, params_lowp=s["copy"],
                               exp_avg_scales=s["ms"] + none, exp_avg_sq_scales=s["vs"] + none)
    s["opt"].step(s["list"], grad_divisor=DIVISOR, max_norm=MAX_NORM)
    return _states(s)


_own = dict(emb_fwd=_own_emb_fwd, emb_bwd=_own_emb_bwd, head_fwd=_own_head_fwd, head_bwd=_own_head_bwd,
            head_loss_grad=_own_head_loss_grad, adamw=_own_adamw)


def _states(s):
    """The updated buffers of a step: an 8-bit moment is its values (e4m3) and its blocks' scales."""
    return {k: s[k] for k in ("small.p", "small.copy", "small.m", "small.ms", "small.v", "small.vs", "whole.p",
                              "whole.copy", "whole.m", "whole.v") if s[k] is not None}


# ---- their plain forms ----------------------------------------------------


def _plain_emb_fwd(s):
    valid = (s["index"] >= 0) & (s["index"] < s["vocab"])
    y = s["table"][torch.where(valid, s["index"], 0).long()].float() * s["scale"]
    return torch.where(valid[:, None], y, 0.0).to(s["table"].dtype)


def _plain_emb_bwd(s):
    valid = (s["index"] >= 0) & (s["index"] < s["vocab"])
    dy = torch.where(valid[:, None], s["dy"].float() * s["scale"], 0.0)
    total = torch.zeros(s["vocab"], s["cols"], device=dy.device)
    total.index_add_(0, torch.where(valid, s["index"], 0).long(), dy)
    if s["out"] is None:
        return total.to(s["dy"].dtype)
    return s["out"].copy_(total.add_(s["out"]))


def _plain_logits(s):
    """Logits, the rows that count and their tokens."""
    counts = (s["row_weight"] != 0) & (s["index"] >= 0) & (s["index"] < s["vocab"])
    z = s["x"].float() @ s["weight"].float().t()
    return z, counts, torch.where(counts, s["index"], 0).long()


def _plain_loss(s, z, counts, at):
    top = z.max(dim=1, keepdim=True).values
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(dim=1))
    loss = s["row_weight"] * (lse - z.gather(1, at[:, None])[:, 0])
    return torch.where(counts, loss, 0.0), torch.where(counts, lse, 0.0)


def _plain_gradients(s, z, lse, scale, counts, at):
    z.sub_(lse[:, None]).exp_()
    z.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    z.mul_(torch.where(counts, scale, 0.0)[:, None])
    dt = s["x"].dtype
    return (z @ s["weight"].float()).to(dt), (z.t() @ s["x"].float()).to(dt)


def _plain_head_fwd(s):
    return _plain_loss(s, *_plain_logits(s))


def _plain_head_bwd(s):
    z, counts, at = _plain_logits(s)
    return _plain_gradients(s, z, s["lse"], s["grad_loss"] * s["row_weight"], counts, at)


def _plain_head_loss_grad(s):
    z, counts, at = _plain_logits(s)
    loss, lse = _plain_loss(s, z, counts, at)
    return (loss, *_plain_gradients(s, z, lse, s["row_weight"], counts, at))


def _random_bits(block, step):
    """32 bits for each element of the blocks: a hash of the element's place in its tensor and the step count."""
    low = 0xffffffff
    i = block[:, None] * BLOCK + torch.arange(BLOCK, device=block.device)
    x = (i & low) ^ (((i >> 32) * 0xc4a8b3f7 + step * 0x9e3779b9) & low)
    x = ((x ^ (x >> 16)) * 0x49a901a7) & low
    x = ((x ^ (x >> 15)) * 0x5fe29a0f) & low
    return (x ^ (x >> 16)).reshape(-1)


def _to_8_bits(x, bits, least):
    """(e4m3 values, scales) of x rounded up or down by chance: `bits` has 16 random bits for each element; what is not 0
    gets at least the code `least`."""
    blocks = x.view(-1, BLOCK)
    top = blocks.abs().max(dim=1, keepdim=True).values
    top = torch.where(top < 2.0 ** -100, 0.0, top)
    y = torch.where(top > 0, blocks.abs() * (TOP / top), 0.0).view(-1)
    # 2^-120 times an e4m3 value has that value's bits, 20 places up
    code = ((y * 2.0 ** -120).view(torch.int32) + (bits.int() * 16 + 8)) >> 20
    code = torch.where(y > 0, code.clamp(least, 126), 0) | torch.where(x < 0, 128, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), (top * (1.0 / TOP))[:, 0]


def _plain_adamw(s):
    total = s["small.g"].double().square().sum() + s["whole.g"].double().square().sum()
    norm = total.sqrt() / DIVISOR
    scale = (torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0) / DIVISOR).float()
    t = s["step"]
    s["step"] = t + 1
    rate, root = LR / (1.0 - BETA1 ** t), 1.0 / math.sqrt(1.0 - BETA2 ** t)

    def step(part, m, v):
        """New weights in place; the moments."""
        g = s[part + ".g"].float() * scale
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + g.square() * (1.0 - BETA2)
        s[part + ".p"].mul_(1.0 - LR * DECAY).sub_(m / (v.sqrt() * root + EPS) * rate)
        if s["masters"]:
            s[part + ".copy"].copy_(s[part + ".p"])
        return m, v

    def values(name):
        return (s["small." + name].float().view(-1, BLOCK) * s[f"small.{name}s"][:, None]).view(-1)
    m, v = step("small", values("m"), values("v").square())
    bits = _random_bits(s["small.block"], t)
    outs = (*_to_8_bits(m, bits & 0xffff, 0), *_to_8_bits(v.sqrt(), bits >> 16, 1))
    s["small.m"].copy_(outs[0]), s["small.ms"].copy_(outs[1]), s["small.v"].copy_(outs[2]), s["small.vs"].copy_(outs[3])
    m, v = step("whole", s["whole.m"], s["whole.v"])
    s["whole.m"].copy_(m), s["whole.v"].copy_(v)
    return _states(s)


_plain = dict(emb_fwd=_plain_emb_fwd, emb_bwd=_plain_emb_bwd, head_fwd=_plain_head_fwd, head_bwd=_plain_head_bwd,
              head_loss_grad=_plain_head_loss_grad, adamw=_plain_adamw)


# ---- the definitions in 64 bits ---------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    v, index = case["vocab"], s["index"].long()
    outside = (index < 0) | (index >= v)
    index = index.clamp(0, v - 1)
    if case["op"] == "emb_fwd":
        return (s["table"].index_select(0, index).double() * case["scale"]).masked_fill(outside.unsqueeze(1), 0.0)
    if case["op"] == "emb_bwd":
        out = torch.zeros(v, case["cols"], device="cuda", dtype=torch.float64)
        kept = torch.nonzero(~outside).squeeze(1)
        for at in range(0, case["cols"], 1024):
            out[:, at:at + 1024].index_put_((index[kept],), s["dy"][kept, at:at + 1024].double() * case["scale"],
                                            accumulate=True)
        return out if s["out"] is None else out + s["out"].double()
    w = s["row_weight"].double().masked_fill(outside, 0.0)
    weight = s["weight"].double()
    losses, lses, dxs, dw = [], [], [], torch.zeros_like(weight) if case["op"] != "head_fwd" else None
    for at in range(0, case["rows"], 1024):
        part = slice(at, at + 1024)
        x, here = s["x"][part].double(), w[part]
        logq = torch.einsum("rk,vk->rv", x, weight)
        lse = s["lse"][part].double() if case["op"] == "head_bwd" else torch.logsumexp(logq, 1)
        logq -= lse.unsqueeze(1)
        losses.append(-here * logq.gather(1, index[part].unsqueeze(1)).squeeze(1))
        lses.append(lse.masked_fill(here == 0, 0.0))
        if dw is not None:
            if case["op"] == "head_bwd":
                here = here * s["grad_loss"][part].double()
            dz = torch.exp(logq) * here.unsqueeze(1)
            dz[torch.arange(len(here), device="cuda"), index[part]] -= here
            dxs.append(dz @ weight)
            dw.addmm_(dz.t(), x)
    if case["op"] == "head_fwd":
        return torch.cat(losses), torch.cat(lses)
    if case["op"] == "head_bwd":
        return torch.cat(dxs), dw
    return torch.cat(losses), torch.cat(dxs), dw


def _exact_adamw(s):
    t = s["step"]
    parts = [s["small.g"].double() / DIVISOR, s["whole.g"].double() / DIVISOR]
    norm = torch.cat(parts).norm()
    clip = min(1.0, MAX_NORM / (norm.item() + 1e-6))
    out = {}
    for part, g in zip(("small", "whole"), parts):
        g = g * clip
        m, v = s[part + ".m"].double(), s[part + ".v"].double()
        if part == "small":
            m = (m.view(-1, BLOCK) * s["small.ms"].double().unsqueeze(1)).flatten()
            v = (v.view(-1, BLOCK) * s["small.vs"].double().unsqueeze(1)).flatten() ** 2
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g * g, v, BETA2)
        mh, vh = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        out[part + ".p"] = s[part + ".p"].double() * (1 - LR * DECAY) - LR * mh / (vh ** 0.5 + EPS)
        if s["masters"]:
            out[part + ".copy"] = out[part + ".p"]
        if part == "whole":
            out["whole.m"], out["whole.v"] = m, v
            continue
        h = _random_bits(s["small.block"], t)  # (the random numbers are part of the definition)
        for name, x, chance in (("m", m, h % 65536), ("v", v ** 0.5, h // 65536)):
            top = x.view(-1, BLOCK).abs().amax(1)
            y = x.abs() / torch.where(top > 0, top / TOP, 1.0).repeat_interleave(BLOCK)
            # the distance of neighbouring e4m3 values around y: an eighth of its power of two, 2^-9 below 2^-6
            gap = torch.exp2(torch.frexp(y.clamp(min=2.0 ** -6)).exponent.double() - 4)
            up = torch.floor(y / gap + (chance.double() + 0.5) / 65536) * gap
            if name == "v":
                up = torch.where(y > 0, up.clamp(min=2.0 ** -9), up)
            out["small." + name] = up.clamp(max=TOP) * torch.sign(x)
            out[f"small.{name}s"] = top / TOP
    return out
