"""Workloads of the operators that train the token decoder: what each computes, in a plain form and by the library's calls.

A decoder that predicts Gaussians from images keeps one token for 256 Gaussians (1k, 100k, 1M and 10M
Gaussians are 4, 391, 3907 and 39063 tokens).  Three operators stand around its attention:

* layer_norm: what each part of a layer starts with, forward and backward, with the gradients of
  weight and bias summed over all rows;
* group_mm: the feed-forward part's products where tokens go to experts: rows sorted by expert, a
  weight for each, ragged numbers of rows; forward, and both gradients;
* adamw: the optimizer's step over all tensors of the decoder, moments in 32 bits or as 8-bit codes.

The codes of adamw: for each 256 units of a tensor, with M and V the block's largest |m| and v (float32),
  m is M (c / 127)^2 with c's sign, c = rint(127 sqrt(|m| / M)); v is V (c / 255)^4, c = rint(255 (v / V)^(1/4)), at least 1 where v > 0.
"""
from __future__ import annotations

import math

import torch

own = False  # True: run() calls the library; False: the plain form

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5
_BLOCK = 256  # units of one pair of bounds
_ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
_DECAY = 0.01


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # four tokens of the example decoder's width before a product: latency
        dict(name="layer-norm-step", op="norm", step=False, type="bf16", rows=4, width=256),
        # training at 1M Gaussians
        dict(name="layer-norm-train", op="norm", step=True, type="bf16", rows=3907, width=2048),
        # training at 10M Gaussians in float32
        dict(name="layer-norm-large-f32", op="norm", step=True, type="f32", rows=39063, width=4096),
        # a few new tokens through eight small experts, most of them without any: latency
        dict(name="experts-tiny", op="group", step=False, type="bf16", rows=6, groups=8, k=256, n=1024, spare=0, layout="kn"),
        # a short batch of tokens through sixteen experts: each weight is read for a handful of rows
        dict(name="experts-few", op="group", step=False, type="bf16", rows=64, groups=16, k=2048, n=4096, spare=0, layout="kn"),
        # training at 100k Gaussians in float32, two experts a token, and padding behind the last one's rows
        dict(name="experts-train-f32", op="group", step=True, type="f32", rows=800, groups=4, k=512, n=1024, spare=18, layout="kn"),
        # a head of odd width for each of five cameras' tokens
        dict(name="experts-odd", op="group", step=True, type="bf16", rows=1955, groups=5, k=363, n=250, spare=3, layout="nk"),
        # training at 1M Gaussians, two experts a token, weights as a linear layer keeps them
        dict(name="experts-train", op="group", step=True, type="bf16", rows=7814, groups=8, k=2048, n=4096, spare=0, layout="nk"),
        # the largest: training at 10M Gaussians, two experts a token, gate and up in one product
        dict(name="experts-train-large", op="group", step=True, type="bf16", rows=78126, groups=16, k=2048, n=8192, spare=0, layout="kn"),
        # the example decoder's ten tensors
        dict(name="adamw-small", op="adamw", bits=8, type="f32", copies=False, tensors=10, units=900_000),
        # a float32 decoder of 48M parameters, moments in 32 bits
        dict(name="adamw-32", op="adamw", bits=32, type="f32", copies=False, tensors=60, units=48_000_000),
        # a bfloat16 decoder of 300M parameters with float32 masters, moments in 8 bits
        dict(name="adamw-large", op="adamw", bits=8, type="bf16", copies=True, tensors=190, units=300_000_000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _even(rng, n):
    """Mostly a multiple of 8, as widths are."""
    return -(-n // 8) * 8 if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["norm", "group", "group", "adamw"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        width = _even(rng, _log(rng, 16, 16000))
        return dict(op=op, step=rng.random() < 0.6, type=kind, rows=min(_log(rng, 1, 60000), 120_000_000 // width), width=width)
    if op == "adamw":
        tensors = _log(rng, 1, 400)
        return dict(op=op, bits=rng.choice([8, 8, 32]), type=kind, copies=rng.random() < 0.5, tensors=tensors, units=max(tensors, _log(rng, 1000, 200_000_000)))
    step = rng.random() < 0.6
    groups, k, n = _log(rng, 1, 64), _even(rng, _log(rng, 32, 6000)), _even(rng, _log(rng, 32, 6000))
    groups = max(1, min(groups, 400_000_000 // (k * n)))
    rows = min(_log(rng, 1, 60000), max(1, int((2e12 if kind == "bf16" else 1e11) / (k * n * (6 if step else 2)))))
    return dict(op=op, step=step, type=kind, rows=rows, groups=groups, k=k, n=n, spare=rng.choice([0, 0, 1, 37]), layout=rng.choice(["kn", "nk"]))


# ---------------------------------------------------------------------------------------------
# sizes that depend on the case alone (so that the work does) and whose order on the seed


def _rows_of(case):
    """Rows of each group: popular ones and others, one without any where there are more than two."""
    g = case["groups"]
    share = [0.0 if g > 2 and i == g - 1 else (1.0 + i) ** -0.5 for i in range(g)]
    whole = sum(share)
    at = [round(case["rows"] * sum(share[: i + 1]) / whole) for i in range(g)]
    return [b - a for a, b in zip([0] + at, at)]


def _units_of(case):
    """Units of each tensor: matrices of a few sizes, and a vector among every four."""
    share = [0.001 if i % 4 == 3 else 1.0 + i % 3 for i in range(case["tensors"])]
    whole = sum(share)
    return [max(1, int(case["units"] * s / whole)) for s in share]


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        return dict(bytes=(4 if case["step"] else 2) * n * size + 16 * case["width"], flops=(25 if case["step"] else 8) * n)
    if case["op"] == "group":
        rows, used = case["rows"], sum(r > 0 for r in _rows_of(case))
        x, y, w = rows * case["k"], rows * case["n"], used * case["k"] * case["n"]
        return dict(bytes=((2 * x + 2 * y + w + case["groups"] * case["k"] * case["n"]) if case["step"] else (x + y + w)) * size,
                    flops=(6 if case["step"] else 2) * rows * case["k"] * case["n"])
    # parameter and moments in and out, the gradient in, the copy out; the values that codes stand for, out
    state = 2 * 8 if case["bits"] == 32 else 2 * 2 + 16 / _BLOCK + 8
    return dict(bytes=int(sum(_units_of(case)) * (8 + size + state + (2 if case["copies"] else 0))), flops=20 * sum(_units_of(case)))


# ---------------------------------------------------------------------------------------------
# inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _generator(seed)
    t = _TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(t)

    s = dict(case=dict(case))
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]
        s.update(x=normal(rows, width, std=1.5).add_(0.3), w=1.0 + 0.2 * torch.randn(width, generator=g, device="cuda"),
                 b=0.1 * torch.randn(width, generator=g, device="cuda"))
        if case["step"]:
            s.update(dy=normal(rows, width, std=0.1))
        return s
    if case["op"] == "group":
        k, n, groups = case["k"], case["n"], case["groups"]
        order = torch.randperm(groups, generator=g, device="cuda").tolist()
        sizes = _rows_of(case)
        ends = [0]
        ends += [sum(sizes[j] for j in order[: i + 1]) for i in range(groups)]
        rows = case["rows"] + case["spare"]
        w = normal(groups, k, n, std=k**-0.5) if case["layout"] == "kn" else normal(groups, n, k, std=k**-0.5).transpose(1, 2)
        s.update(x=normal(rows, k), w=w, offsets=torch.tensor(ends, dtype=torch.int32, device="cuda"), ends=ends)
        if case["step"]:
            s.update(dy=normal(rows, n, std=0.1))
        return s
    units = _units_of(case)
    at = [0]
    at += [sum(-(-u // _BLOCK) * _BLOCK for u in units[: i + 1]) for i in range(len(units))]
    flat, grad = torch.zeros(at[-1], device="cuda"), torch.zeros(at[-1], dtype=t, device="cuda")
    copy = torch.zeros(at[-1], dtype=torch.bfloat16, device="cuda") if case["copies"] else None
    # vectors (one tensor of four) are not decayed; every tensor is a view of one buffer, as the example decoder's are
    decay = [0.0 if i % 4 == 3 else _DECAY for i in range(len(units))]
    views = [slice(a, a + u) for a, u in zip(at, units)]
    for i, v in enumerate(views):
        std = 0.02 * (1 + i % 5)
        flat[v].normal_(0.0, std, generator=g)
        # gradients of very different sizes within a block, as rows of a weight have
        grad[v].copy_(torch.randn(units[i], generator=g, device="cuda").pow_(3).mul_(1e-3 * (1 + i % 3)))
    s.update(flat=flat, grad=grad, copy=copy, step=10, params=[flat[v] for v in views], grads=[grad[v] for v in views],
             copies=[copy[v] for v in views] if case["copies"] else None, decay=decay,
             decays=torch.tensor([d for d, u in zip(decay, units) for _ in range(-(-u // _BLOCK))], dtype=torch.float64, device="cuda"))
    # moments that earlier steps left
    m = torch.zeros_like(flat)
    for v in views:
        m[v].normal_(0.0, 1.0, generator=g).pow_(3).mul_(5e-4)
    v = (m * 2).square_().add_(m.abs().mul_(1e-6))
    if case["bits"] == 32:
        s.update(m=m, v=v, bounds=None)
    else:
        codes = _encode(m.double(), v.double())
        s.update(m=codes[0], v=codes[1], bounds=codes[2])
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    c = s["case"]
    if own:
        from tile_differentiable_rasterizer_amd import tokens

        if c["op"] == "norm":
            y = tokens.layer_norm_fwd(s["x"], s["w"], s["b"], eps=_EPS)
            return [y, tokens.layer_norm_bwd(s["dy"], s["x"], s["w"], eps=_EPS)] if c["step"] else y
        if c["op"] == "group":
            y = tokens.group_mm_fwd(s["x"], s["w"], s["offsets"])
            return [y, tokens.group_mm_bwd(s["dy"], s["x"], s["w"], s["offsets"])] if c["step"] else y
        state = tokens.AdamWState(s["m"], s["v"], s["bounds"])
        tokens.adamw(s["params"], s["grads"], state, step=s["step"], weight_decay=s["decay"], copies=s["copies"], **_ADAM)
        s["step"] += 1
        out = [s["flat"], *tokens.adamw_moments(state)]
        return out + [s["copy"]] if c["copies"] else out
    return {"norm": _norm, "group": _group, "adamw": _adamw}[c["op"]](s)


def _norm(s):
    t, x, w = s["x"].dtype, s["x"].float(), s["w"]
    d = x - x.mean(-1, keepdim=True)
    rstd = (d.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    xh = d * rstd
    y = (xh * w + s["b"]).to(t)
    if not s["case"]["step"]:
        return y
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return [y, (dx.to(t), (dy * xh).sum(0), dy.sum(0))]


def _group(s):
    """The rows that belong to no group (behind the last one's) are 0, in the result and in the gradient."""
    t, x, w, ends = s["x"].dtype, s["x"], s["w"], s["ends"]
    parts = [slice(a, b) for a, b in zip(ends, ends[1:])]

    def behind(width):
        return torch.zeros(x.shape[0] - ends[-1], width, device="cuda", dtype=t)

    y = torch.cat([torch.matmul(x[p].float(), w[i].float()).to(t) for i, p in enumerate(parts)] + [behind(w.shape[2])])
    if not s["case"]["step"]:
        return y
    dy = s["dy"]
    dx = torch.cat([torch.matmul(dy[p].float(), w[i].float().t()).to(t) for i, p in enumerate(parts)] + [behind(w.shape[1])])
    # as the weights lie: their last two axes may be exchanged
    if s["case"]["layout"] == "kn":
        dw = torch.stack([torch.matmul(x[p].float().t(), dy[p].float()).to(t) for p in parts])
    else:
        dw = torch.stack([torch.matmul(dy[p].float().t(), x[p].float()).to(t) for p in parts]).transpose(1, 2)
    return [y, (dx, dw)]


def _decode(m, v, bounds):
    """Moments in 64 bits from their codes, whole blocks."""
    top = bounds.double()
    c, e = m.view(-1, _BLOCK).double(), v.view(-1, _BLOCK).double()
    return ((top[:, :1] / 127.0**2) * c * c.abs()).view(-1), ((top[:, 1:] / 255.0**4) * e.pow(4)).view(-1)


def _encode(m, v):
    """Codes and bounds of moments in 64 bits: values next to a border between two codes are decided there."""
    m, v = m.view(-1, _BLOCK), v.view(-1, _BLOCK)
    top = torch.stack([m.abs().amax(1), v.amax(1)], 1).float()
    inv = torch.where(top > 0, 1.0 / top.double(), torch.zeros_like(top, dtype=torch.float64))
    c = (m.abs() * inv[:, :1]).sqrt().mul(127.0).round().clamp(max=127.0) * m.sign()
    e = (v * inv[:, 1:]).sqrt().sqrt().mul(255.0).round().clamp(max=255.0)
    e = torch.where(v > 0, e.clamp(min=1.0), e) * (top[:, 1:] > 0)
    return c.to(torch.int8).view(-1), e.to(torch.uint8).view(-1), top


def _adamw(s):
    c, h = s["case"], _ADAM
    g = s["grad"].double()
    if c["bits"] == 8:
        m, v = _decode(s["m"], s["v"], s["bounds"])
    else:
        m, v = s["m"].double(), s["v"].double()
    m = m.mul_(h["beta1"]).add_(g, alpha=1.0 - h["beta1"])
    v = v.mul_(h["beta2"]).add_(g.square_(), alpha=1.0 - h["beta2"])
    step = m / (1.0 - h["beta1"] ** s["step"]) / ((v / (1.0 - h["beta2"] ** s["step"])).sqrt_() + h["eps"])
    p = s["flat"].view(-1, _BLOCK).double().mul_(1.0 - h["lr"] * s["decays"][:, None]).view(-1)
    s["flat"].copy_(p.sub_(step, alpha=h["lr"]))
    s["step"] += 1
    if c["copies"]:
        s["copy"].copy_(s["flat"])
    if c["bits"] == 8:
        codes = _encode(m, v)
        s["m"].copy_(codes[0])
        s["v"].copy_(codes[1])
        s["bounds"].copy_(codes[2])
        m, v = _decode(s["m"], s["v"], s["bounds"])
        out = [s["flat"], m.float(), v.float()]
    else:
        out = [s["flat"], s["m"].copy_(m), s["v"].copy_(v)]
    return out + [s["copy"]] if c["copies"] else out


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    if not torch.cuda.is_available() and work(case)["flops"] > 1e10:
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, w, b = (s[n].double().requires_grad_(case["step"]) for n in ("x", "w", "b"))
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + _EPS) * w + b
        if not case["step"]:
            return y
        return [y.detach(), torch.autograd.grad(y, (x, w, b), s["dy"].double())]
    if case["op"] == "group":
        edge = s["offsets"].tolist()
        x, w = s["x"].double(), s["w"].double()
        y = torch.zeros(x.shape[0], case["n"], dtype=torch.float64, device="cuda")
        for i in range(case["groups"]):
            y[edge[i]: edge[i + 1]] = x[edge[i]: edge[i + 1]] @ w[i]
        if not case["step"]:
            return y
        dy = s["dy"].double()
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        for i in range(case["groups"]):
            at = slice(edge[i], edge[i + 1])
            dx[at] = dy[at] @ w[i].mT
            dw[i] = x[at].mT @ dy[at]
        return [y, (dx, dw)]
    f = lambda x: x.double()  # noqa: E731
    if case["bits"] == 8:
        blocks = s["bounds"].shape[0]
        m = (f(s["m"]).view(blocks, -1) / 127.0).mul_(f(s["m"]).abs().view(blocks, -1) / 127.0).mul_(f(s["bounds"][:, :1])).view(-1)
        v = (f(s["v"]).view(blocks, -1) / 255.0).pow_(4).mul_(f(s["bounds"][:, 1:])).view(-1)
    else:
        m, v = f(s["m"]), f(s["v"])
    g, t = f(s["grad"]), s["step"]
    m = torch.lerp(g, m, _ADAM["beta1"])
    v = torch.lerp(g * g, v, _ADAM["beta2"])
    ratio = (m / (1 - _ADAM["beta1"] ** t)).div_((v / (1 - _ADAM["beta2"] ** t)).sqrt_().add_(_ADAM["eps"]))
    p = f(s["flat"])
    p = p - _ADAM["lr"] * (ratio + s["decays"].repeat_interleave(_BLOCK) * p)
    del g, ratio
    if case["bits"] == 8:
        def stored(x, levels, power, floor):
            x = x.view(-1, _BLOCK)
            top = x.abs().amax(1, keepdim=True).float().double()
            code = torch.nan_to_num((x.abs() / top) ** (1.0 / power) * levels).round().clamp(0, levels)
            if floor:
                code = torch.where(x != 0, code.clamp(min=1), code)
            return ((code / levels) ** power * top * x.sign()).view(-1)

        m, v = stored(m, 127, 2, False), stored(v, 255, 4, True)
    return [p, m, v, p] if case["copies"] else [p, m, v]
