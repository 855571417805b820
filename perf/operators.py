"""The token operators' workloads: what each case computes, in a plain form and by the library's calls.

A decoder that predicts Gaussians from images keeps one token for 256 Gaussians (so 1k, 100k, 1M and
10M Gaussians are 4, 391, 3907 and 39063 tokens) and lets them attend to one encoder state for each
16x16 tile of the cameras' images (16 at 64x64, 2500 at 800x800, 3600 at 1280x720, 8160 at 1920x1080,
65280 for eight cameras).  Three operators make up its layer:

* norm_rotate: RMS norm of each head's query and key vector, weight, and the position rotation;
* cross_attn: attention of the tokens to the states, with shared heads, a key range for each
  query row and a mask byte for each key;
* gate8: the feed-forward part's gated activation, its inputs kept as 8-bit codes for the backward pass.
"""
from __future__ import annotations

import math

import torch

own = False  # True: run() calls the library; False: the plain form

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_BLOCK = 256  # units of one (lo, hi) pair of gate8's codes
_GELU = math.sqrt(2.0 / math.pi)


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one new Gaussian token and the states of one 64x64 image: latency
        dict(name="norm-step", op="norm", step=False, type="bf16", batch=1, lq=1, lk=16, hq=8, hk=2, d=64, rot=64, pairs="halves"),
        # training at 100k Gaussians, four cameras of 800x800, half of each head rotated, neighbouring pairs
        dict(name="norm-train", op="norm", step=True, type="bf16", batch=4, lq=391, lk=2500, hq=16, hk=4, d=128, rot=64, pairs="neighbours"),
        # 10M Gaussians and eight 1080p cameras in float32, a head size that is no power of two
        dict(name="norm-large-f32", op="norm", step=True, type="f32", batch=1, lq=39063, lk=65280, hq=16, hk=16, d=96, rot=96, pairs="halves"),
        # 1k Gaussians against one 64x64 image: latency
        dict(name="attend-tiny", op="attend", step=False, type="bf16", batch=1, lq=4, lk=16, hq=8, hk=8, d=64, mask="none"),
        # one token for each of eight sequences, 1080p states of ragged length (one of them empty)
        dict(name="attend-token", op="attend", step=False, type="bf16", batch=8, lq=1, lk=8160, hq=32, hk=4, d=128, mask="lens"),
        # 1M Gaussians against eight 1080p cameras, each run of tokens seeing some of the cameras (some none)
        dict(name="attend-views", op="attend", step=False, type="bf16", batch=1, lq=3907, lk=65280, hq=16, hk=4, d=64, mask="views"),
        # training at 100k Gaussians in float32, states with holes
        dict(name="attend-train-f32", op="attend", step=True, type="f32", batch=2, lq=391, lk=2500, hq=8, hk=8, d=64, mask="keys"),
        # training at 1M Gaussians, three 720p cameras as sequences of ragged length
        dict(name="attend-train", op="attend", step=True, type="bf16", batch=3, lq=3907, lk=3600, hq=16, hk=16, d=64, mask="lens"),
        # the largest training step: 1M Gaussians, two 1080p cameras, shared heads
        dict(name="attend-train-large", op="attend", step=True, type="bf16", batch=2, lq=3907, lk=8160, hq=32, hk=8, d=128, mask="none"),
        # a few tokens through the feed-forward part, an odd width: latency
        dict(name="gate-small", op="gate", type="bf16", rows=4, width=1001, act="gelu"),
        # training at 1M Gaussians
        dict(name="gate-train", op="gate", type="bf16", rows=3907, width=4096, act="silu"),
        # training at 10M Gaussians in float32, a width that is no multiple of a code block
        dict(name="gate-large-f32", op="gate", type="f32", rows=39063, width=2752, act="silu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "attend", "attend", "gate"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "gate":
        width = _log(rng, 200, 5000)
        if rng.random() < 0.7:
            width = -(-width // 8) * 8
        return dict(op=op, type=kind, rows=_log(rng, 1, 20000), width=width, act=rng.choice(["silu", "gelu"]))
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 4])
    d = rng.choice([32, 64, 64, 80, 96, 128, 128])
    if op == "norm":
        rot = rng.choice([d, d, d // 2 // 8 * 8])
        return dict(op=op, step=rng.random() < 0.5, type=kind, batch=rng.randint(1, 3), lq=_log(rng, 1, 8000), lk=_log(rng, 1, 8160), hq=hq, hk=hk,
                    d=d, rot=rot, pairs=rng.choice(["halves", "neighbours"]))
    step = rng.random() < 0.5
    batch, lk = rng.randint(1, 4), _log(rng, 1, 65280 if kind == "bf16" else 8160)
    most = (4e11 if kind == "bf16" else 2e10) / (batch * hq * lk * d * (14 if step else 4))
    lq = min(_log(rng, 1, 4000), max(1, int(most)))
    return dict(op=op, step=step, type=kind, batch=batch, lq=lq, lk=lk, hq=hq, hk=hk, d=d, mask=rng.choice(["none", "lens", "views", "keys"]))


# ---------------------------------------------------------------------------------------------
# the masks, whose sizes depend on the case alone (so that the work does) and whose order on the seed


def _spans(case):
    """The key ranges of the case, (rows that share one, [lengths]): by sequence, or by runs of query rows."""
    b, lq, lk = case["batch"], case["lq"], case["lk"]
    if case["mask"] == "lens":  # full, down to a quarter, and one empty where there are more than two
        n = [max(1, round(lk * (1.0 - 0.75 * i / max(1, b - 1)))) for i in range(b)]
        if b > 2:
            n[-1] = 0
        return lq, n
    run = 192  # neighbouring tokens see the same cameras
    runs = b * -(-lq // run)
    return run, [max(1, lk * (1 + i % 4) // 4) if i % 8 != 7 else 0 for i in range(runs)]


def _pairs(case):
    """(row, key) pairs that the masks allow, over all query heads."""
    b, lq, lk, hq = case["batch"], case["lq"], case["lk"], case["hq"]
    if case["mask"] in ("none", "keys"):
        return b * lq * (lk if case["mask"] == "none" else lk - lk // 4) * hq
    if case["mask"] == "lens":
        return sum(_spans(case)[1]) * lq * hq
    n = _spans(case)[1]
    return round(sum(n) / len(n) * b * lq) * hq


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "gate":
        n = case["rows"] * case["width"]
        codes = 2 * n + 16 * case["rows"] * -(-case["width"] // _BLOCK)
        # forward: gate and up in, y and codes out; backward: codes and dy in, dgate, dup and y again out
        return dict(bytes=3 * n * size + codes + codes + 4 * n * size, flops=40 * n)
    b, lq, lk, hq, hk, d = (case[k] for k in ("batch", "lq", "lk", "hq", "hk", "d"))
    nq, nk = b * lq * hq * d, b * lk * hk * d
    if case["op"] == "norm":
        passes = 5 if case["step"] else 2  # x in, y out; and x and dy in, dx out
        return dict(bytes=passes * (nq + nk) * size + 4 * max(lq, lk) * case["rot"], flops=(30 if case["step"] else 10) * (nq + nk))
    moved = (2 * nq + 2 * nk) + ((4 * nq + 4 * nk) if case["step"] else 0)
    return dict(bytes=moved * size + 4 * b * lq * hq, flops=_pairs(case) * d * (14 if case["step"] else 4))


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _generator(seed)
    t = _TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)

    def weight(n):
        return 1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")

    s = dict(case=dict(case))
    if case["op"] == "gate":
        # gate and up are the two halves of one projection's output, as the product leaves them
        h = normal(case["rows"], 2 * case["width"], std=1.5)
        s.update(gate=h[:, : case["width"]], up=h[:, case["width"]:], dy=normal(case["rows"], case["width"], std=0.1))
        return s
    b, lq, lk, hq, hk, d = (case[k] for k in ("batch", "lq", "lk", "hq", "hk", "d"))
    s.update(q=normal(b, lq, hq, d, std=1.3))
    kv = normal(b, lk, 2, hk, d)  # keys and values of one projection, interleaved
    s.update(k=kv[:, :, 0], v=kv[:, :, 1])
    if case["op"] == "norm":
        half = case["rot"] // 2
        n = max(lq, lk)
        angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s.update(wq=weight(d), wk=weight(d), cos=angle.cos().float(), sin=angle.sin().float())
        # a token's place: the states in order, the queries at places of their own
        s.update(pos_q=torch.randint(0, n, (b, lq), generator=g, device="cuda", dtype=torch.int32), pos_k=None)
        if case["step"]:
            s.update(dq=normal(b, lq, hq, d, std=0.1), dk=normal(b, lk, hk, d, std=0.1))
        return s
    s.update(ranges=None, mask=None, scale=d**-0.5)
    if case["mask"] in ("lens", "views"):
        run, n = _spans(case)
        n = torch.tensor(n, device="cuda")[torch.randperm(len(n), generator=g, device="cuda")]
        if case["mask"] == "lens":
            s["ranges"] = torch.stack([torch.zeros_like(n), n], 1).int().view(b, 1, 2)
        else:
            first = torch.minimum((torch.rand(n.shape, generator=g, device="cuda") * (lk - n + 1)).long(), lk - n)
            r = torch.stack([first, first + n], 1).view(b, -1, 2)
            s["ranges"] = r.repeat_interleave(run, 1)[:, :lq].int().contiguous()
    if case["mask"] == "keys":  # a quarter of the states carry nothing, in runs of up to 16
        order = torch.rand(b, -(-lk // 16), generator=g, device="cuda").repeat_interleave(16, 1)[:, :lk]
        at = order.argsort(dim=1, stable=True)[:, : lk // 4]
        s["mask"] = torch.ones(b, lk, dtype=torch.uint8, device="cuda").scatter_(1, at, 0)
    if case["step"]:
        s["dout"] = normal(b, lq, hq, d, std=0.1)
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    c = s["case"]
    if own:
        from tile_differentiable_rasterizer_amd import tokens

        if c["op"] == "norm":
            args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"])
            more = dict(pos_q=s["pos_q"], pos_k=s["pos_k"], eps=_EPS, pairs=c["pairs"])
            out = tokens.norm_rotate_fwd(*args, **more)
            return [out, tokens.norm_rotate_bwd(s["dq"], s["dk"], *args, **more)] if c["step"] else out
        if c["op"] == "attend":
            more = dict(scale=s["scale"], ranges=s["ranges"], key_mask=s["mask"])
            out, lse = tokens.cross_attn_fwd(s["q"], s["k"], s["v"], **more)
            return [out, lse, tokens.cross_attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, **more)] if c["step"] else [out, lse]
        y, codes, bounds = tokens.gate8_fwd(s["gate"], s["up"], act=c["act"])
        return [y, tokens.gate8_bwd(s["dy"], codes, bounds, act=c["act"])]
    return {"norm": _norm, "attend": _attend, "gate": _gate}[c["op"]](s)


def _halves(x, rot, pairs):
    """The rotated elements' pairs as (a, b)."""
    return (x[..., : rot // 2], x[..., rot // 2: rot]) if pairs == "halves" else (x[..., 0:rot:2], x[..., 1:rot:2])


def _whole(a, b, rest, pairs):
    return torch.cat([a, b, rest], -1) if pairs == "halves" else torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _norm_one(x, w, cos, sin, dy, c):
    t, x = x.dtype, x.float()
    rot = c["rot"]
    rstd = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    xh = x * rstd
    y = xh * w
    a, b = _halves(y, rot, c["pairs"])
    y = _whole(a * cos - b * sin, a * sin + b * cos, y[..., rot:], c["pairs"]).to(t)
    if dy is None:
        return y, None, None
    dy = dy.float()
    a, b = _halves(dy, rot, c["pairs"])
    g = _whole(a * cos + b * sin, b * cos - a * sin, dy[..., rot:], c["pairs"])
    dw = (g * xh).sum((0, 1, 2))
    g = g * w
    return y, (rstd * (g - xh * (g * xh).mean(-1, keepdim=True))).to(t), dw


def _norm(s):
    c = s["case"]
    at = s["pos_q"].long()
    n = c["lk"]
    y_q, dq, dwq = _norm_one(s["q"], s["wq"], s["cos"][at][:, :, None], s["sin"][at][:, :, None], s.get("dq"), c)
    y_k, dk, dwk = _norm_one(s["k"], s["wk"], s["cos"][None, :n, None], s["sin"][None, :n, None], s.get("dk"), c)
    return [(y_q, y_k), (dq, dk, dwq, dwk)] if c["step"] else (y_q, y_k)


def _allowed(s, lk):
    """Truth values [batch, 1, rows, keys] (rows 1 where every row has the same)."""
    ok = None
    if s["ranges"] is not None:
        at = torch.arange(lk, device="cuda", dtype=torch.int32)
        ok = (at >= s["ranges"][..., :1]) & (at < s["ranges"][..., 1:])
    if s["mask"] is not None:
        ok = s["mask"][:, None] != 0
    return None if ok is None else ok[:, None]


def _attend(s):
    c = s["case"]
    b, lq, lk, hq, hk, d = (c[k] for k in ("batch", "lq", "lk", "hq", "hk", "d"))
    t, group = s["q"].dtype, hq // hk

    def by_head(x):  # [batch, heads, tokens, d] in 32 bits
        return x.float().transpose(1, 2).contiguous()

    def shared(x):  # the query heads of one key head after one another: [batch, hk, group * lq, d]
        return by_head(x).view(b, hk, group * lq, d)

    def back(x, heads, n):
        return x.reshape(b, heads, n, d).transpose(1, 2).to(t)

    q, k, v = shared(s["q"]), by_head(s["k"]), by_head(s["v"])
    p = torch.matmul(q, k.transpose(-1, -2)).view(b, hq, lq, lk) * s["scale"]
    ok = _allowed(s, lk)
    if ok is not None:
        p = p.masked_fill_(~ok, -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total)).view(b, hk, group * lq, lk)
    o = torch.matmul(p, v)
    out = back(o, hq, lq).contiguous()
    if not c["step"]:
        return [out, lse]
    do = shared(s["dout"])
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dv = torch.matmul(p.transpose(-1, -2), do)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    return [out, lse, (back(dq, hq, lq).contiguous(), back(dk, hk, lk).contiguous(), back(dv, hk, lk).contiguous())]


def _act(x, kind):
    """The activation and its derivative."""
    if kind == "silu":
        h = 1.0 / (1.0 + (-x).exp())
        return x * h, h * (1.0 + x * (1.0 - h))
    th = (_GELU * (x + 0.044715 * x * x * x)).tanh()
    return 0.5 * x * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * x * (1.0 - th * th) * (_GELU * (1.0 + 3 * 0.044715 * x * x))


def _kept(x):
    """What the 8-bit codes of x stand for.  The definition decides a code in 64 bits, so that nothing hangs on rounding."""
    rows, width = x.shape
    fill = -width % _BLOCK
    x = torch.cat([x, x[:, -1:].expand(rows, fill)], 1).view(rows, -1, _BLOCK) if fill else x.reshape(rows, -1, _BLOCK)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    span = hi.double() - lo.double()
    code = ((x.double() - lo.double()) * torch.where(span > 0, 255.0 / span, torch.zeros_like(span))).round()
    return (lo + code.float() * ((hi - lo) * (1.0 / 255.0))).view(rows, -1)[:, :width]


def _gate(s):
    c = s["case"]
    t = s["gate"].dtype
    g, u, dy = s["gate"].float(), s["up"].float(), s["dy"].float()
    y = (_act(g, c["act"])[0] * u).to(t)
    # the last block of a row holds fewer units: the row's last value again changes no minimum and no maximum
    g, u = _kept(g), _kept(u)
    a, da = _act(g, c["act"])
    return [y, ((dy * u * da).to(t), (dy * a).to(t), (a * u).to(t))]


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    if not torch.cuda.is_available() and work(case)["flops"] > 1e10:
        return None
    s = prepare(case, seed)
    c = s["case"]
    f = lambda x: x.double()  # noqa: E731
    if c["op"] == "gate":
        g, u, dy = f(s["gate"]), f(s["up"]), f(s["dy"])
        act = torch.nn.functional.silu if c["act"] == "silu" else lambda x: torch.nn.functional.gelu(x, approximate="tanh")

        def stored(x):
            parts = []
            for part in x.split(_BLOCK, 1):
                lo, hi = part.amin(1, keepdim=True), part.amax(1, keepdim=True)
                code = torch.nan_to_num((part - lo) * (255.0 / (hi - lo))).round().clamp(0, 255)
                parts.append(lo + code * (hi - lo) / 255.0)
            return torch.cat(parts, 1)

        y = act(g) * u
        gs, us = stored(g).requires_grad_(), stored(u).requires_grad_()
        again = act(gs) * us
        dg, du = torch.autograd.grad(again, (gs, us), dy)
        return [y, (dg, du, again.detach())]
    if c["op"] == "norm":
        wq, wk = f(s["wq"]).requires_grad_(), f(s["wk"]).requires_grad_()
        q, k = f(s["q"]).requires_grad_(), f(s["k"]).requires_grad_()
        turn = torch.complex(f(s["cos"]), f(s["sin"]))

        def one(x, w, turns):
            y = x * w / (x.pow(2).mean(-1, keepdim=True) + _EPS).sqrt()
            head, rest = y[..., : c["rot"]], y[..., c["rot"]:]
            if c["pairs"] == "halves":
                z = torch.complex(*head.chunk(2, -1)) * turns
                return torch.cat([z.real, z.imag, rest], -1)
            z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turns
            return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)

        with torch.set_grad_enabled(c["step"]):
            yq = one(q, wq, turn[s["pos_q"].long()].unsqueeze(2))
            yk = one(k, wk, turn[: c["lk"]].unsqueeze(1))
        if not c["step"]:
            return (yq, yk)
        grads = torch.autograd.grad((yq, yk), (q, k, wq, wk), (f(s["dq"]), f(s["dk"])))
        return [(yq.detach(), yk.detach()), grads]
    group = c["hq"] // c["hk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["batch"], c["hq"], c["lq"], dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (s["q"], s["k"], s["v"]))
    keys = torch.arange(c["lk"], device="cuda")
    for i in range(c["batch"]):
        seen = torch.ones(1, c["lk"], dtype=torch.bool, device="cuda")
        if s["ranges"] is not None:
            seen = (keys >= s["ranges"][i, :, :1]) & (keys < s["ranges"][i, :, 1:])
        if s["mask"] is not None:
            seen = seen & s["mask"][i].bool()
        for h in range(c["hq"]):
            q, k, v = f(s["q"][i, :, h]), f(s["k"][i, :, h // group]), f(s["v"][i, :, h // group])
            score = torch.where(seen, q @ k.T * s["scale"], -math.inf)
            lse[i, h] = score.logsumexp(-1)
            p = torch.nan_to_num((score - lse[i, h][:, None]).exp())
            out[i, :, h] = p @ v
            if c["step"]:
                do = f(s["dout"][i, :, h])
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
                dq[i, :, h] = ds @ k
                dk[i, :, h // group] += ds.T @ q
                dv[i, :, h // group] += p.T @ do
    return [out, lse, (dq, dk, dv)] if c["step"] else [out, lse]
