"""GPU tests of the token operators against plain implementations in 64 bits, at the sizes, strides
and masks where they can go wrong.

Tolerances follow from what the kernels round, u = 2^-24 (float32) and v = 2^-8 (bfloat16: half a
spacing, 8 significant bits), and are taken element by element from the reference's own sums of absolute values (and 2^-120 for what underflows):

* norm_rotate: a vector's sum of squares over D elements, a square root, a division and five more
  products: (D / 8 + 16) u of the largest terms of an output; bfloat16 outputs are rounded once more.
* cross_attn: a score's error is (D + 8) u of sum |q| |k| |scale|, and a weight's relative error
  e = 2 times that (its own and the sum's) + (keys / 64 + 32) u for the exponentials and the sum;
  weights and score gradients enter products as elements (v in bfloat16, u in float32).  So
  out: (e + v) sum p |v_j| + v |out|; dv: the same with the kept lse; ds: p (e |dp - delta| +
  e_dp + e_delta) + v |ds|, where e_delta holds out's own error, and dq, dk the products of that.
* gate8: codes and bounds exactly; values within 16 u relative of the float64 formula on the decoded
  values (plus the formula's own slope where 1 - h cancels), and v in bfloat16.
"""
import math

import pytest
import torch

from tile_differentiable_rasterizer_amd import raster, tokens

pytestmark = pytest.mark.gpu

U, V, TINY = 2.0**-24, 2.0**-8, 2.0**-120
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, t=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)


def half_step(t):
    return V if t == torch.bfloat16 else U


def close(got, want, tol, what):
    """|got - want| <= tol, element by element; not-finite places must agree."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), what + ": places that are not finite"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    over = ((got - want).abs() - tol)[fine] - TINY
    assert not (over > 0).any(), f"{what}: {int((over > 0).sum())} of {over.numel()} off, worst by {over.max().item():.3e}"


# -- norm with rotation ------------------------------------------------------------------------


def norm_ref(x, w, cos, sin, eps, pairs, dy=None):
    """float64: y, and (dx, dw) where dy is given; the sums of absolute terms of each."""
    x, w = x.double(), w.double()
    D, half = x.shape[-1], cos.shape[-1]
    rot = 2 * half
    rstd = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    xh = x * rstd
    y = xh * w
    ia = torch.arange(half, device=x.device)
    ia, ib = (ia, ia + half) if pairs == "halves" else (2 * ia, 2 * ia + 1)
    c, s = cos.double(), sin.double()
    out, mag = y.clone(), y.abs()
    out[..., ia] = y[..., ia] * c - y[..., ib] * s
    out[..., ib] = y[..., ia] * s + y[..., ib] * c
    both = (y[..., ia].abs() + y[..., ib].abs()) if rot else y[..., :0]
    mag[..., ia] = both
    mag[..., ib] = both
    if dy is None:
        return out, mag
    dy = dy.double()
    g, gm = dy.clone(), dy.abs()
    g[..., ia] = dy[..., ia] * c + dy[..., ib] * s
    g[..., ib] = dy[..., ib] * c - dy[..., ia] * s
    both = dy[..., ia].abs() + dy[..., ib].abs()
    gm[..., ia] = both
    gm[..., ib] = both
    dw, dwm = (g * xh).sum((0, 1, 2)), (gm * xh.abs()).sum((0, 1, 2))
    gw, gwm = g * w, gm * w.abs()
    dx = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    dxm = rstd * (gwm + xh.abs() * (gwm * xh.abs()).mean(-1, keepdim=True))
    return out, mag, dx, dxm, dw, dwm


NORMS = [  # type, batch, lq, lk, hq, hk, d, rot, pairs
    ("bf16", 1, 1, 16, 8, 2, 64, 64, "halves"), ("f32", 1, 1, 1, 1, 1, 8, 8, "neighbours"),
    ("bf16", 2, 37, 5, 3, 1, 8, 0, "halves"), ("bf16", 3, 11, 23, 4, 2, 16, 8, "neighbours"),
    ("f32", 2, 9, 31, 5, 5, 40, 24, "halves"), ("bf16", 2, 64, 33, 6, 3, 96, 96, "halves"),
    ("f32", 1, 129, 77, 4, 4, 128, 64, "neighbours"), ("bf16", 1, 50, 70, 2, 1, 136, 136, "halves"),
    ("f32", 2, 21, 13, 3, 2, 256, 256, "halves"), ("bf16", 2, 19, 40, 16, 4, 256, 128, "neighbours"),
    ("bf16", 2, 3000, 2500, 8, 8, 64, 64, "halves"), ("f32", 1, 0, 17, 4, 4, 64, 64, "halves"), ("bf16", 1, 17, 0, 4, 4, 64, 32, "halves"),
]


def norm_inputs(case, strided):
    t, B, lq, lk, hq, hk, d, rot, pairs = case
    t, g = TYPES[t], gen(17)
    if strided:  # heads before tokens, and a projection's interleaved parts
        q = normal(g, B, hq, lq, d + 16, t=t).transpose(1, 2)[..., 8: 8 + d]
        k = normal(g, B, lk, 2, hk, d, t=t)[:, :, 1]
    else:
        q, k = normal(g, B, lq, hq, d, t=t), normal(g, B, lk, hk, d, t=t)
    n = max(lq, lk) + 3
    ang = torch.rand(n, rot // 2, generator=g, device="cuda") * 6.28
    return q, k, normal(g, d) + 1, normal(g, d) + 1, ang.cos(), ang.sin()


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("case", NORMS, ids=str)
def test_norm_rotate(case, strided):
    pairs = case[-1]
    q, k, wq, wk, cos, sin = norm_inputs(case, strided)
    g, n = gen(3), cos.shape[0]
    pos_q = torch.randint(0, n, q.shape[:2], generator=g, device="cuda", dtype=torch.int32) if strided else None
    args = (q, k, wq, wk, cos, sin, pos_q, None, 1e-5, pairs)
    yq, yk = tokens.norm_rotate_fwd(*args)
    dyq, dyk = normal(g, *q.shape, t=q.dtype), normal(g, *k.shape, t=k.dtype)
    dq, dk, dwq, dwk = tokens.norm_rotate_bwd(dyq, dyk, *args)
    again = tokens.norm_rotate_bwd(dyq, dyk, *args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again)), "the same bits on every call"
    e, r = (q.shape[-1] / 8 + 16) * U, half_step(q.dtype)
    for x, w, y, dy, dx, dw, pos, side in ((q, wq, yq, dyq, dq, dwq, pos_q, "q"), (k, wk, yk, dyk, dk, dwk, None, "k")):
        at = pos.long() if pos is not None else torch.arange(x.shape[1], device="cuda")[None]
        out, mag, rx, rxm, rw, rwm = norm_ref(x, w, cos[at][:, :, None], sin[at][:, :, None], 1e-5, pairs, dy)
        close(y, out, e * mag + r * out.abs(), side)
        close(dx, rx, 2 * e * rxm + r * rx.abs(), "d" + side)
        terms = x.shape[0] * x.shape[1] * x.shape[2]  # a lane's chain, then lanes, wavefronts and workgroups
        close(dw, rw, (e + (terms / 2048 + 64) * U) * rwm, "dw" + side)


def test_norm_rotate_more_vectors_than_a_grid_takes():
    """Workgroups walk the vectors: forward from 65536 workgroups on, back with more parts of dw than 2048."""
    test_norm_rotate(("bf16", 1, 40000, 1000, 16, 4, 256, 64, "halves"), False)


def test_norm_rotate_in_place_and_positions_outside_the_table():
    q, k, wq, wk, cos, sin = norm_inputs(("bf16", 2, 33, 12, 4, 2, 64, 64, "halves"), False)
    n = cos.shape[0]
    pos = torch.randint(-5, n + 5, q.shape[:2], generator=gen(1), device="cuda", dtype=torch.int32)
    pos[0, 0], pos[0, 1] = -(2**31), 2**31 - 1
    want = tokens.norm_rotate_fwd(q, k, wq, wk, cos, sin, pos.clamp(0, n - 1), None)
    qc, kc = q.clone(), k.clone()
    got = tokens.norm_rotate_fwd(qc, kc, wq, wk, cos, sin, pos, None, out=(qc, kc))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0] is qc


def test_norm_rotate_zero_and_infinite_vectors():
    q, k, wq, wk, cos, sin = norm_inputs(("f32", 1, 6, 6, 1, 1, 64, 0, "halves"), False)
    q[0, 0] = 0
    q[0, 1, 0, 5] = float("nan")
    q[0, 2, 0, 7] = float("inf")
    yq, yk = tokens.norm_rotate_fwd(q, k, wq, wk, cos, sin)
    assert (yq[0, 0] == 0).all() and yq[0, 1].isnan().all() and yq[0, 2, 0, 7].isnan() and torch.isfinite(yq[0, 3:]).all()


def differences(loss, x, u, h):
    """The derivative of loss along u by differences of fourth order."""
    f = lambda s: loss((x.double() + s * h * u.double()).float()).item()  # noqa: E731
    return (8 * (f(1) - f(-1)) - (f(2) - f(-2))) / (12 * h)


def test_norm_rotate_against_differences():
    # h^4 of the fifth derivative (below 1 for unit vectors) plus float32 values' noise over h
    q, k, wq, wk, cos, sin = norm_inputs(("f32", 2, 9, 7, 3, 2, 32, 16, "neighbours"), False)
    g = gen(8)
    dyq, dyk = normal(g, *q.shape), normal(g, *k.shape)

    def loss(i):
        def f(x):
            a = [q, k, wq, wk]
            a[i] = x
            yq, yk = tokens.norm_rotate_fwd(*a, cos, sin, pairs="neighbours")
            return (yq.double() * dyq).sum() + (yk.double() * dyk).sum()
        return f

    grads = tokens.norm_rotate_bwd(dyq, dyk, q, k, wq, wk, cos, sin, pairs="neighbours")
    for i, x in enumerate((q, k, wq, wk)):
        u = normal(g, *x.shape)
        u /= u.norm()
        h = 0.03
        want = differences(loss(i), x, u, h)
        size = math.sqrt(dyq.numel() + dyk.numel())
        assert abs((grads[i].double() * u).sum().item() - want) <= 4 * h**4 + 64 * U * size / h, i


# -- cross attention ---------------------------------------------------------------------------


def seen_of(B, Lq, Lk, ranges, mask):
    ok = torch.ones(B, Lq, Lk, dtype=torch.bool, device="cuda")
    at = torch.arange(Lk, device="cuda")
    if ranges is not None:
        r = ranges.long().expand(B, Lq, 2)
        ok &= (at >= r[..., :1]) & (at < r[..., 1:])
    if mask is not None:
        ok &= (mask != 0)[:, None]
    return ok


def attn_ref(q, k, v, scale, ranges, mask, dout=None, out=None):
    """float64 by (batch, head), with the tolerances: dict name -> (value, tolerance)."""
    t = q.dtype
    e_el = half_step(t) * 1.01
    B, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1:3]
    G = Hq // Hk
    ok = seen_of(B, Lq, Lk, ranges, mask)
    o, to = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse, tl = (torch.zeros(B, Hq, Lq, dtype=torch.float64, device="cuda") for _ in range(2))
    gq, tq = torch.zeros_like(o), torch.zeros_like(o)
    gk, tk, gv, tv = (torch.zeros(k.shape, dtype=torch.float64, device="cuda") for _ in range(4))
    for b in range(B):
        hidden = ~ok[b].any(0)  # keys that no row sees: whatever they hold
        for h in range(Hq):
            Q, K, Vv = q[b, :, h].double(), k[b, :, h // G].double(), v[b, :, h // G].double()
            K, Vv = K.masked_fill(hidden[:, None], 0), Vv.masked_fill(hidden[:, None], 0)
            dead = ~ok[b].any(1)
            Q = Q.masked_fill(dead[:, None], 0)
            s = (Q @ K.T * scale).masked_fill(~ok[b], -math.inf)
            es = (D + 8) * U * abs(scale) * (Q.abs() @ K.abs().T)
            es = es.masked_fill(~ok[b], 0).amax(1, keepdim=True) if Lk else es.sum(1, keepdim=True)
            e = 2 * es + (Lk / 64 + 32) * U
            lse[b, h] = s.logsumexp(1) if Lk else -math.inf
            tl[b, h] = (e + 4 * U * lse[b, h][:, None].abs().nan_to_num(0, 0, 0))[:, 0]
            p = (s - lse[b, h][:, None]).exp().nan_to_num(0, 0, 0)
            o[b, :, h] = p @ Vv
            to[b, :, h] = (e + e_el) * (p @ Vv.abs()) + e_el * o[b, :, h].abs()
            if dout is None:
                continue
            dO = dout[b, :, h].double().masked_fill(dead[:, None], 0)
            dp = dO @ Vv.T
            delta = (dO * o[b, :, h]).sum(1, keepdim=True)
            e_delta = (dO.abs() * to[b, :, h]).sum(1, keepdim=True) + (D + 8) * U * (dO * o[b, :, h]).abs().sum(1, keepdim=True)
            e_dp = (D + 8) * U * (dO.abs() @ Vv.abs().T)
            e2 = e + 8 * U + 4 * U * (s.nan_to_num(0, 0, 0).abs() + lse[b, h][:, None].nan_to_num(0, 0, 0).abs())
            ds = p * (dp - delta)
            eds = p * (e2 * (dp - delta).abs() + e_dp + e_delta) + e_el * ds.abs()
            more = (max(Lq * G, Lk) / 32 + 32) * U  # a sum's own additions
            gq[b, :, h] = scale * ds @ K
            tq[b, :, h] = abs(scale) * ((eds + more * ds.abs()) @ K.abs())
            gk[b, :, h // G] += scale * ds.T @ Q
            tk[b, :, h // G] += abs(scale) * ((eds + more * ds.abs()).T @ Q.abs())
            gv[b, :, h // G] += p.T @ dO
            tv[b, :, h // G] += ((e2 + e_el + more) * p).T @ dO.abs()
    res = {"out": (o, to), "lse": (lse, tl)}
    if dout is not None:
        res.update(dq=(gq, tq + e_el * gq.abs()), dk=(gk, tk + e_el * gk.abs()), dv=(gv, tv + e_el * gv.abs()))
    return res


def attn_check(q, k, v, scale=None, ranges=None, mask=None, bwd=True, seed=2):
    scale = q.shape[3] ** -0.5 if scale is None else scale
    out, lse = tokens.cross_attn_fwd(q, k, v, scale, ranges, mask)
    got = {"out": out, "lse": lse}
    dout = normal(gen(seed), *q.shape, t=q.dtype) if bwd else None
    if bwd:
        got.update(zip(("dq", "dk", "dv"), tokens.cross_attn_bwd(dout, q, k, v, out, lse, scale, ranges, mask)))
        again = tokens.cross_attn_bwd(dout, q, k, v, out, lse, scale, ranges, mask)
        assert all(torch.equal(a, b) for a, b in zip((got["dq"], got["dk"], got["dv"]), again)), "the same bits on every call"
    for name, (want, tol) in attn_ref(q, k, v, scale, ranges, mask, dout).items():
        close(got[name], want, tol, name)
    return got


def qkv(t, B, Lq, Lk, Hq, Hk, D, seed=5):
    g = gen(seed)
    return normal(g, B, Lq, Hq, D, t=TYPES[t]), normal(g, B, Lk, Hk, D, t=TYPES[t]), normal(g, B, Lk, Hk, D, t=TYPES[t])


ATTNS = [  # type, batch, lq, lk, hq, hk, d
    ("bf16", 1, 1, 1, 1, 1, 64), ("f32", 1, 1, 1, 2, 1, 8), ("bf16", 2, 3, 2, 2, 2, 8), ("bf16", 1, 4, 16, 8, 8, 64), ("f32", 1, 31, 33, 3, 1, 24),
    ("bf16", 2, 32, 64, 4, 2, 32), ("bf16", 1, 33, 65, 6, 3, 40), ("f32", 2, 64, 63, 2, 2, 64), ("bf16", 1, 127, 129, 4, 1, 96), ("f32", 1, 65, 190, 2, 1, 96),
    ("bf16", 1, 200, 300, 4, 4, 128), ("f32", 1, 140, 200, 4, 2, 128), ("bf16", 3, 5, 700, 10, 2, 72), ("bf16", 4, 1, 3001, 8, 1, 128), ("f32", 3, 1, 1500, 4, 2, 64),
    ("bf16", 2, 2, 5000, 4, 4, 64), ("bf16", 1, 3000, 16, 2, 2, 64), ("f32", 1, 1500, 7, 2, 1, 32), ("bf16", 1, 700, 900, 2, 2, 112), ("bf16", 1, 513, 64, 12, 4, 16),
    ("bf16", 2, 0, 9, 2, 1, 64), ("bf16", 2, 9, 0, 2, 1, 64), ("f32", 0, 4, 4, 2, 1, 64),
]


@pytest.mark.parametrize("case", ATTNS, ids=str)
def test_cross_attn(case):
    attn_check(*qkv(*case))


def bad_places(x, where, value):
    x[where] = value
    return x


@pytest.mark.parametrize("case", [("bf16", 3, 70, 333, 4, 2, 64), ("f32", 3, 70, 200, 2, 2, 32), ("bf16", 3, 1, 2000, 8, 2, 128), ("bf16", 3, 300, 90, 4, 4, 96)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), None])
def test_cross_attn_lengths(case, value):
    """Lengths of sequences, one of them 0 and one 1; what lies past them is not part of any result."""
    q, k, v = qkv(*case)
    Lk = k.shape[1]
    n = torch.tensor([0, 1, Lk - 5], device="cuda")
    ranges = torch.stack([torch.zeros_like(n), n], 1).int()[:, None]
    fill = torch.finfo(k.dtype).min if value is None else value
    past = torch.arange(Lk, device="cuda") >= n[:, None]
    bad_places(k, past, fill)
    bad_places(v, past, fill)
    q[0] = float("nan")  # a sequence without keys
    got = attn_check(q, k, v, ranges=ranges)
    assert (got["out"][0] == 0).all() and (got["lse"][0] == -math.inf).all()
    assert (got["dq"][0] == 0).all() and (got["dk"][0] == 0).all() and (got["dv"][0] == 0).all()


@pytest.mark.parametrize("case", [("bf16", 2, 300, 500, 4, 2, 64), ("f32", 2, 150, 260, 4, 1, 40), ("bf16", 1, 7, 4000, 4, 2, 128), ("bf16", 2, 2000, 130, 2, 2, 32)], ids=str)
def test_cross_attn_row_ranges(case):
    """A range for each row: empty, reversed, past both ends, one key, ends inside tiles; gaps that no row sees hold NaN."""
    q, k, v = qkv(*case)
    B, Lq, Lk = q.shape[0], q.shape[1], k.shape[1]
    g = gen(11)
    a = torch.randint(-20, Lk + 20, (B, Lq), generator=g, device="cuda")
    n = torch.randint(-3, Lk // 2, (B, Lq), generator=g, device="cuda")
    n[:, ::5] = 1
    n[:, 1::7] = 0
    ranges = torch.stack([a, a + n], -1).int()
    gap = slice(Lk // 3, Lk // 3 + 30)  # nobody sees these
    lo, hi = ranges[..., 0], ranges[..., 1]
    cut = lo < gap.start
    ranges[..., 1] = torch.where(cut, hi.clamp(max=gap.start), hi)
    ranges[..., 0] = torch.where(cut, lo, lo.clamp(min=gap.stop))
    k[:, gap] = float("nan")
    v[:, gap] = float("nan")
    attn_check(q, k, v, ranges=ranges)


@pytest.mark.parametrize("case", [("bf16", 2, 1300, 2600, 8, 8, 32), ("f32", 2, 2000, 1100, 8, 8, 32), ("f32", 1, 900, 1500, 16, 8, 104)], ids=str)
@pytest.mark.parametrize("kind", ["all", "rows", "lengths"])
def test_cross_attn_many_blocks(case, kind):
    """Enough workgroups for a part of the GPU or for more than it holds: long axes in a few parts."""
    q, k, v = qkv(*case)
    B, Lq, Lk = q.shape[0], q.shape[1], k.shape[1]
    ranges = None
    if kind == "rows":
        first = torch.randint(0, Lk, (B, Lq), generator=gen(13), device="cuda")
        ranges = torch.stack([first, first + torch.randint(0, Lk, (B, Lq), generator=gen(14), device="cuda")], -1).int()
    if kind == "lengths":
        ranges = torch.tensor([[0, Lk - 70], [65, 67]], device="cuda", dtype=torch.int32)[:B, None]
    attn_check(q, k, v, ranges=ranges)


@pytest.mark.parametrize("kind", ["rows", "lengths"])
def test_cross_attn_longest_first(kind):
    """From 2^28 pairs on, blocks of rows with ranges are worked on by length."""
    q, k, v = qkv("bf16", 2, 4200, 2100, 16, 16, 32)
    p = tokens.GsCrossAttn(2, 4200, 2100, 16, 16, 32, tokens.BF16, 1.0)
    plain = tokens.lib().gs_cross_attn_fwd_workspace_bytes(p)
    p.ranges, p.ranges_batch_stride = 1 << 20, 1
    assert tokens.lib().gs_cross_attn_fwd_workspace_bytes(p) > plain  # room for the order
    if kind == "lengths":
        ranges = torch.tensor([[[3, 1000]], [[0, 2100]]], device="cuda", dtype=torch.int32)
    else:
        first = torch.randint(0, 2000, (2, 4200 // 60, 1), generator=gen(15), device="cuda").expand(-1, -1, 60).reshape(2, -1)
        n = torch.randint(0, 2100, (2, 4200 // 60, 1), generator=gen(16), device="cuda").expand(-1, -1, 60).reshape(2, -1)
        ranges = torch.stack([first, first + n], -1).int().contiguous()
    attn_check(q, k, v, ranges=ranges)


def test_cross_attn_extreme_ranges():
    q, k, v = qkv("bf16", 1, 6, 70, 2, 2, 64)
    big = 2**31 - 1
    r = torch.tensor([[0, big], [-big - 1, big], [big, big], [-big - 1, -5], [69, big], [64, 3]], device="cuda", dtype=torch.int32)[None]
    attn_check(q, k, v, ranges=r)


@pytest.mark.parametrize("case", [("bf16", 2, 90, 400, 4, 4, 64), ("f32", 2, 40, 130, 2, 1, 64), ("bf16", 2, 1, 3000, 4, 1, 128)], ids=str)
@pytest.mark.parametrize("kind", ["random", "all", "none", "tail", "with ranges"])
def test_cross_attn_key_mask(case, kind):
    q, k, v = qkv(*case)
    B, Lk = k.shape[:2]
    g = gen(4)
    mask = torch.rand(B, Lk, generator=g, device="cuda") < 0.6
    if kind == "all":
        mask[0] = False  # rows of sequence 0 see nothing
    if kind == "none":
        mask[:] = True
    if kind == "tail":
        mask[:, Lk // 2:] = False
    k[~mask] = float("nan")
    v[~mask] = float("inf")
    ranges = None
    if kind == "with ranges":
        a = torch.randint(0, Lk, (1, q.shape[1]), generator=g, device="cuda")
        ranges = torch.stack([a, a + Lk // 4], -1).int()
    wide = torch.zeros(B, Lk + 5, dtype=torch.uint8, device="cuda")
    wide[:, :Lk] = mask.to(torch.uint8) * 7
    attn_check(q, k, v, ranges=ranges, mask=wide[:, :Lk])


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("lq", [1, 45])
def test_cross_attn_strides(t, lq):
    """Heads before tokens, interleaved keys and values, one key sequence for the whole batch, padded vectors."""
    g, t = gen(6), TYPES[t]
    q = normal(g, 2, 6, lq, 64 + 8, t=t).transpose(1, 2)[..., :64]
    kv = normal(g, 1, 310, 2, 3, 64, t=t)
    k, v = kv[:, :, 0].expand(2, -1, -1, -1), kv[:, :, 1].expand(2, -1, -1, -1)
    attn_check(q, k, v)
    attn_check(q, normal(g, 2, 3, 200, 64, t=t).transpose(1, 2), normal(g, 2, 200, 3, 80, t=t)[..., 16:])


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_cross_attn_scales(scale):
    """Flat, negative and steep weights (one key takes all)."""
    q, k, v = qkv("f32", 1, 40, 150, 2, 2, 32)
    attn_check(q, k, v, scale=scale)
    q, k, v = qkv("bf16", 1, 40, 150, 2, 2, 64)
    attn_check(q, k, v, scale=scale)


def test_cross_attn_scores_that_fall_and_rise():
    """The running maximum rises by hundreds late in the row, or never after the first tile."""
    for order in (1, -1):
        q, k, v = qkv("bf16", 1, 70, 640, 2, 2, 64)
        k *= (torch.linspace(0, 8, 640, device="cuda")[::1] if order == 1 else torch.linspace(8, 0, 640, device="cuda"))[None, :, None, None].to(k.dtype)
        q = q.abs() * (1 if order == 1 else 1)
        attn_check(q, k, v, scale=0.5)


def test_cross_attn_nan_reaches_only_its_own():
    """A NaN in one query or one seen key shows where the formula has it and nowhere else."""
    q, k, v = qkv("f32", 2, 40, 100, 2, 2, 64)
    q[0, 3, 1] = float("nan")
    out, lse = tokens.cross_attn_fwd(q, k, v)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 3, 1] = True
    assert torch.equal(out.isnan(), bad) and torch.equal(lse.isnan(), bad[..., 0].transpose(1, 2))


def test_cross_attn_against_differences():
    # h^4 of the fifth derivative plus float32 values' noise over h, as above
    q, k, v = qkv("f32", 2, 9, 70, 4, 2, 32)
    g = gen(9)
    dout = normal(g, *q.shape)
    ranges = torch.tensor([[[0, 70]], [[3, 40]]], dtype=torch.int32, device="cuda")

    def loss(i):
        def f(x):
            a = [q, k, v]
            a[i] = x
            return (tokens.cross_attn_fwd(*a, ranges=ranges)[0].double() * dout).sum()
        return f

    out, lse = tokens.cross_attn_fwd(q, k, v, ranges=ranges)
    grads = tokens.cross_attn_bwd(dout, q, k, v, out, lse, ranges=ranges)
    for i, x in enumerate((q, k, v)):
        u = normal(g, *x.shape)
        u /= u.norm()
        h = 0.03
        want = differences(loss(i), x, u, h)
        assert abs((grads[i].double() * u).sum().item() - want) <= 16 * h**4 + 64 * U * math.sqrt(dout.numel()) / h, i


def test_cross_attn_far_offsets():
    """Keys and values whose last elements lie past 2^32 bytes and past 2^31 elements from their base."""
    g = gen(13)
    base = torch.empty((1, 2**31 // 512 + 300, 1, 512), dtype=torch.bfloat16, device="cuda")
    n = base.shape[1]
    base[:, :200] = 0
    k = base[:, n - 290::, :, :64]  # the view starts past 2^31 elements
    k.copy_(normal(g, *k.shape, t=torch.bfloat16))
    far = torch.as_strided(base, (1, 3, 1, 64), (0, (n - 1) // 2 * 512, 512, 1))  # three keys 2^30 elements apart
    far.copy_(normal(g, 1, 3, 1, 64, t=torch.bfloat16))
    q = normal(g, 1, 5, 2, 64, t=torch.bfloat16)
    attn_check(q, k, k)
    attn_check(q, far, far)


def test_tokens_on_another_stream():
    """Calls on a stream of their own, inputs made on it, results waited for there."""
    side = torch.cuda.Stream()
    want = None
    for _ in range(3):
        with torch.cuda.stream(side):
            q, k, v = qkv("bf16", 2, 100, 3000, 4, 2, 64)
            out, lse = tokens.cross_attn_fwd(q, k, v)
            grads = tokens.cross_attn_bwd(out, q, k, v, out, lse)
        side.synchronize()
        got = [out, lse, *grads]
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
    q, k, v = qkv("bf16", 2, 100, 3000, 4, 2, 64)
    ref = tokens.cross_attn_fwd(q, k, v)
    assert torch.equal(ref[0], want[0]) and torch.equal(ref[1], want[1])


def test_tokens_stream_argument():
    """Work on a stream given by argument while the current one allocates and overwrites: what the calls allocate
    belongs to their stream."""
    side = torch.cuda.Stream()
    q, k, v = qkv("bf16", 2, 40, 6000, 4, 2, 64)
    w, cs = torch.ones(64, device="cuda"), torch.ones(6000, 32, device="cuda")
    h = normal(gen(2), 500, 600, t=torch.bfloat16)

    def step(stream):
        a, b = tokens.norm_rotate_fwd(q, k, w, w, cs, cs, stream=stream)
        out, lse = tokens.cross_attn_fwd(a, b, v, stream=stream)
        grads = tokens.cross_attn_bwd(out, a, b, v, out, lse, stream=stream)
        more = tokens.norm_rotate_bwd(grads[0], grads[1], q, k, w, w, cs, cs, stream=stream)
        y, codes, bounds = tokens.gate8_fwd(h[:, :300], h[:, 300:], stream=stream)
        return [out, lse, *grads, *more, y, *tokens.gate8_bwd(y, codes, bounds, stream=stream)]

    want = step(None)
    torch.cuda.synchronize()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk


def test_tokens_in_a_graph():
    """A captured layer step replays to the eager results, with other work between the replays."""
    q, k, v = qkv("bf16", 2, 3, 2000, 4, 2, 64)
    h = normal(gen(2), 6, 2 * 300, t=torch.bfloat16)
    w, cs = torch.ones(64, device="cuda"), torch.zeros(2000, 32, device="cuda")

    def step():
        a, b = tokens.norm_rotate_fwd(q, k, w, w, cs + 1, cs)
        out, lse = tokens.cross_attn_fwd(a, b, v)
        grads = tokens.cross_attn_bwd(out, a, b, v, out, lse)
        y, codes, bounds = tokens.gate8_fwd(h[:, :300], h[:, 300:])
        return [a, b, out, lse, *grads, y, *tokens.gate8_bwd(y, codes, bounds)]

    for _ in range(2):
        want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(4):
        q.copy_(normal(gen(50 + n), *q.shape, t=q.dtype))
        want = [x.clone() for x in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


# -- gated activation with 8-bit checkpoints ---------------------------------------------------


def gate_codes_ref(x):
    """codes, bounds and decoded values (float32, every operation rounded) by the definition."""
    rows, width = x.shape
    nb = (width + 255) // 256
    x = x.float()
    codes = torch.zeros(rows, width, dtype=torch.uint8, device="cuda")
    bounds = torch.zeros(rows, nb, 2, device="cuda")
    for i in range(nb):
        part = x[:, 256 * i: 256 * (i + 1)]
        lo, hi = part.amin(1), part.amax(1)
        bad = ~torch.isfinite(part).all(1)
        lo, hi = lo.masked_fill(bad, math.nan), hi.masked_fill(bad, math.nan)
        bounds[:, i, 0], bounds[:, i, 1] = lo, hi
        span = (hi.double() - lo.double())[:, None]
        c = (part.double() - lo.double()[:, None]) * (255.0 * (1.0 / span))
        codes[:, 256 * i: 256 * (i + 1)] = torch.where(span > 0, c, torch.zeros_like(c)).round().to(torch.uint8)
    step = (bounds[..., 1] - bounds[..., 0]) * (1.0 / 255.0)
    up = lambda b: b.repeat_interleave(256, 1)[:, :width]  # noqa: E731
    return codes, bounds, up(bounds[..., 0]) + codes.float() * up(step)


def act_ref(x, act):
    x = x.double()
    if act == "silu":
        h = torch.sigmoid(x)
        return x * h, h * (1 + x * (1 - h))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (x + 0.044715 * x**3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * 0.044715 * x * x)


def act_tol(x, act):
    """Error of act and act' in float32: 16 roundings' worth, the exponent's argument |z| U in both, through slopes of at most |x| z'."""
    x = x.double().abs().clamp(max=32)
    z = 2 * x if act == "silu" else 2 * x * (1 + 0.05 * x * x)
    slope = 1 if act == "silu" else 1 + 0.2 * x * x
    return (16 + 4 * z) * U * (1 + x) * slope


GATES = [("bf16", 1, 1, "silu", 0), ("f32", 3, 7, "gelu", 0), ("bf16", 4, 1001, "gelu", 0), ("bf16", 5, 256, "silu", 0), ("f32", 2, 257, "silu", 0),
         ("bf16", 130, 520, "gelu", 0), ("f32", 65, 1024, "gelu", 0), ("bf16", 17, 776, "silu", 8), ("bf16", 17, 776, "silu", 1), ("f32", 9, 300, "silu", 3), ("bf16", 9, 248, "gelu", 16)]


@pytest.mark.parametrize("case", GATES, ids=str)
def test_gate8(case):
    t, rows, width, act, pad = case
    t, g = TYPES[t], gen(21)
    h = normal(g, rows, 2 * width + pad, t=t, std=2.0)
    gate, up = h[:, :width], h[:, width: 2 * width] if pad != 1 else h[:, width + 1:]
    gate[rows // 2, : min(width, 256)] = 0.75  # a constant block
    y, codes, bounds = tokens.gate8_fwd(gate, up, act)
    dy = normal(g, rows, width, t=t)
    r = half_step(t)
    a, _ = act_ref(gate, act)
    want = a * up.double()
    close(y, want, act_tol(gate, act) * up.double().abs() + r * want.abs(), "y")
    gc, gb, gv = gate_codes_ref(gate)
    uc, ub, uv = gate_codes_ref(up)
    assert torch.equal(codes[0], gc) and torch.equal(codes[1], uc)
    assert torch.equal(bounds[0], gb) and torch.equal(bounds[1], ub)
    assert ((gv - gate.float()).abs() <= (gb[..., 1] - gb[..., 0]).amax(1, keepdim=True) / 509).all()
    dg, du, again = tokens.gate8_bwd(dy, codes, bounds, act)
    a, da = act_ref(gv, act)
    d, u, e = dy.double(), uv.double(), act_tol(gv, act)
    for got, want, tol, what in ((dg, d * u * da, e * (d * u).abs(), "dgate"), (du, d * a, e * d.abs(), "dup"), (again, a * u, e * u.abs(), "y again")):
        close(got, want, tol + r * want.abs(), what)
    wide = torch.empty(rows, 2 * width, dtype=t, device="cuda")
    tokens.gate8_bwd(dy, codes, bounds, act, False, wide[:, :width], wide[:, width:])
    assert torch.equal(wide[:, :width], dg) and torch.equal(wide[:, width:], du)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_gate8_extremes(t):
    """Blocks with a NaN or an infinity decode as NaN and leave their neighbours alone; the widest ranges and the
    smallest spans code as any other."""
    t = TYPES[t]
    x = normal(gen(1), 8, 768, t=t)
    top = torch.finfo(t).max
    x[0, 3], x[1, 300], x[2, 767] = math.nan, math.inf, -math.inf
    x[3, :256] = torch.where(torch.arange(256, device="cuda") % 2 == 0, top, -top).to(t)
    x[4, :256] = 1.0
    x[4, 7] = 1.0 + 2.0**-7
    x[5, :256] = 0
    x[5, 9] = 1e-38
    x[6, :256] = -0.0
    up = normal(gen(2), 8, 768, t=t)
    y, codes, bounds = tokens.gate8_fwd(x, up, "silu")
    gc, gb, gv = gate_codes_ref(x)
    assert torch.equal(codes[0], gc)
    assert torch.equal(bounds[0].nan_to_num(7.0), gb.nan_to_num(7.0)) and int(bounds[0].isnan().any(-1).sum()) == 3
    dy = torch.ones(8, 768, dtype=t, device="cuda")
    for act in ("silu", "gelu"):
        dg, du, again = tokens.gate8_bwd(dy, codes, bounds, act)
        lost = torch.zeros(8, 768, dtype=torch.bool, device="cuda")
        lost[0, :256] = lost[1, 256:512] = lost[2, 512:] = True
        if t == torch.float32:
            lost[3, :256] = True  # hi - lo is no float32
        else:
            lost[3, :256] = True
        assert torch.equal(dg.isnan(), lost) and torch.equal(du.isnan() | ~torch.isfinite(du), lost)


def test_gate8_against_differences():
    # through the codes the step is flat: differences of the formula at the decoded values (16 bits would
    # not show it), on a grid where the decoded values are the inputs
    lo, hi = -2.0, 2.0
    g = gen(3)
    code = torch.randint(0, 256, (4, 512), generator=g, device="cuda")
    code[:, 0], code[:, 1], code[:, 256], code[:, 257] = 0, 255, 0, 255
    x = (lo + code.float() * ((hi - lo) * (1.0 / 255.0)))
    x[code == 255] = hi
    up, dy = normal(g, 4, 512), normal(g, 4, 512)
    for act in ("silu", "gelu"):
        _, codes, bounds = tokens.gate8_fwd(x, x, act)
        dg, du, y = tokens.gate8_bwd(dy, codes, bounds, act)
        f = lambda s: tokens.gate8_fwd(x + s, x, act)[0].double()  # noqa: E731
        h = 0.05
        slope = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
        # the fifth derivative of either is below 4; values of up to 4 with 8 roundings over h; decoded values U off
        assert ((dg.double() - dy * slope).abs() <= dy.abs() * (4 * 2 * h**4 + 64 * U / h)).all()
        f = lambda s: tokens.gate8_fwd(x, x + s, act)[0].double()  # noqa: E731
        assert ((du.double() - dy * (f(h) - f(-h)) / (2 * h)).abs() <= dy.abs() * 64 * U / h).all()


# -- as torch functions, and together ----------------------------------------------------------


def test_functions_differentiate():
    g = gen(31)
    q, k, v = (x.requires_grad_() for x in qkv("f32", 2, 20, 50, 4, 2, 32))
    w = (normal(g, 32) + 1).requires_grad_()
    ang = torch.rand(50, 16, generator=g, device="cuda")
    a, b = tokens.norm_rotate(q, k, w, w, ang.cos(), ang.sin())
    out = tokens.cross_attention(a, b, v)
    h = out.reshape(40, 128)
    tokens.gated8(torch.cat([h, h.flip(1)], 1)).sum().backward()
    assert all(x.grad is not None and torch.isfinite(x.grad).all() and x.grad.abs().max() > 0 for x in (q, k, v, w))
    q2 = q.detach().clone().requires_grad_()
    tokens.cross_attention(q2, k.detach(), v.detach()).sum().backward()  # an expanded gradient
    assert torch.isfinite(q2.grad).all()


def test_errors_name_the_call():
    q, k, v = qkv("bf16", 1, 4, 4, 2, 2, 64)
    with pytest.raises(raster.GsError, match="gs_cross_attn_fwd"):
        tokens.cross_attn_fwd(q, k, v, scale=math.nan)
    with pytest.raises(raster.GsError):  # a view that is off its 16-byte boundary
        tokens.cross_attn_fwd(normal(gen(1), 1, 4, 2, 68, t=torch.bfloat16)[..., 1:65], k, v)
    with pytest.raises(raster.GsError, match="workspace"):
        big = qkv("bf16", 1, 1, 9000, 1, 1, 64)
        tokens.cross_attn_fwd(*big, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tokens.cross_attn_fwd(q, k, v, ranges=torch.zeros(1, 3, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        tokens.cross_attn_fwd(q, k, v.float())
    with pytest.raises(ValueError):
        tokens.cross_attn_fwd(q, k.transpose(2, 3), v.transpose(2, 3))


def test_gate8_more_blocks_than_a_grid_axis_takes():
    """2^27 rows and some, a block each: the grid is folded, and every row is worked on."""
    rows, g = 2**27 + 5, gen(41)
    t = torch.bfloat16
    gate, up, dy = (torch.empty((rows, 1), dtype=t, device="cuda").normal_(generator=g) for _ in range(3))
    y, codes, bounds = tokens.gate8_fwd(gate, up)
    dg, du, again = tokens.gate8_bwd(dy, codes, bounds)
    assert not codes.any()
    for i, x in enumerate((gate, up)):  # a block of one unit is its own minimum and maximum
        assert torch.equal(bounds[i, :, 0, 0], x[:, 0].float()) and torch.equal(bounds[i, :, 0, 1], x[:, 0].float())
    assert torch.equal(y, again)
    for part in torch.arange(rows, device="cuda").split(2**24):
        part = slice(int(part[0]), int(part[-1]) + 1)
        a, da = act_ref(gate[part], "silu")
        d, u, e = dy[part].double(), up[part].double(), act_tol(gate[part], "silu")
        for got, want, tol, what in ((dg, d * u * da, e * (d * u).abs(), "dgate"), (du, d * a, e * d.abs(), "dup"), (y, a * u, e * u.abs(), "y")):
            close(got[part], want, tol + V * want.abs(), what)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_functions_take_gradients_off_their_boundaries(t):
    """The gradient of a part of a cat starts at an odd element: the same results as from an aligned one."""
    q, k, v = (x.requires_grad_() for x in qkv(t, 2, 20, 50, 4, 2, 64))
    w, cs = torch.ones(64, device="cuda").requires_grad_(), torch.ones(50, 32, device="cuda")
    first = torch.zeros(1, device="cuda", dtype=q.dtype)

    def parts(*xs):
        """Each tensor's gradient is a part of a larger one, from its second element on where `first` comes before it."""
        return sum((torch.cat([first, x.flatten()])[1:] * x.detach().flatten().flip(0)).sum() for x in xs)

    def grads(loss):
        return torch.autograd.grad(loss, (q, k, v, w), allow_unused=True)

    a, b = tokens.norm_rotate(q, k, w, w, cs, cs)
    out = tokens.cross_attention(q, k, v)
    got, want = grads(parts(a, b)), grads(sum((x.flatten() * x.detach().flatten().flip(0)).sum() for x in tokens.norm_rotate(q, k, w, w, cs, cs)))
    assert all(torch.equal(x, y) for x, y in zip(got, want) if x is not None) and got[3] is not None
    got = grads(parts(out))
    out = tokens.cross_attention(q, k, v)
    want = grads((out.flatten() * out.detach().flatten().flip(0)).sum())
    assert all(torch.equal(x, y) for x, y in zip(got[:3], want[:3]))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("scale, std", [(0.0, 1e16), (-0.0, 1e15), (1e-33, 3e16), (-1e-33, 3e16), (3e-39, 1e18), (1e35, 1e-18)])
def test_cross_attn_scales_for_large_and_small_vectors(t, scale, std):
    """No scale is too small for some finite scores: 0 makes them all 0 whatever the vectors' size, others their own."""
    q, k, v = qkv(t, 2, 40, 150, 4, 2, 64)
    q, k = q * std, k * std
    ranges = torch.tensor([[[0, 150]], [[20, 90]]], device="cuda", dtype=torch.int32)
    mask = torch.rand(2, 150, generator=gen(4), device="cuda") < 0.7
    attn_check(q, k, v, scale=scale, ranges=ranges, mask=mask)


def test_cross_attn_scale_of_nothing_keeps_nan():
    """0 times a NaN or an infinity is a NaN, in the rows that hold it or see it and in no others."""
    for t in ("f32", "bf16"):
        q, k, v = qkv(t, 2, 40, 100, 2, 2, 64)
        q[0, 3, 1, 5], q[0, 7, 0, 0] = math.nan, math.inf
        k[1, 50, 0, 9] = math.inf
        bad = torch.zeros(2, 2, 40, dtype=torch.bool, device="cuda")
        bad[0, 1, 3] = bad[0, 0, 7] = bad[1, 0] = True
        out, lse = tokens.cross_attn_fwd(q, k, v, scale=0.0)
        assert torch.equal(lse.isnan(), bad) and torch.equal(out.isnan().all(-1).transpose(1, 2), bad) and torch.equal(out.isnan().any(-1).transpose(1, 2), bad)
        assert ((lse - math.log(100))[~bad].abs() < 1e-5).all()


# -- the torch functions' gradients are the calls' own -------------------------------------------


def same(got, want):
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b), i


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_norm_rotate_function(t, pairs):
    q, k, wq, wk, cos, sin = norm_inputs((t, 2, 20, 33, 4, 2, 64, 32, pairs), True)
    n, g = cos.shape[0], gen(3)
    pos_q, pos_k = (torch.randint(0, n, x.shape[:2], generator=g, device="cuda", dtype=torch.int32) for x in (q, k))
    more = (cos, sin, pos_q, pos_k, 1e-2, pairs)
    dq, dk = normal(g, *q.shape, t=q.dtype), normal(g, *k.shape, t=k.dtype)
    xs = [x.detach().requires_grad_() for x in (q, k, wq, wk)]
    out = tokens.norm_rotate(*xs, *more)
    same(out, tokens.norm_rotate_fwd(q, k, wq, wk, *more))
    want = tokens.norm_rotate_bwd(dq, dk, q, k, wq, wk, *more)
    assert not torch.equal(want[2], want[3])
    same(torch.autograd.grad(out, xs, (dq, dk)), want)
    out = tokens.norm_rotate(*xs, *more)  # one output used alone
    got = torch.autograd.grad(out[1], xs, dk)
    same((got[1], got[3]), (want[1], want[3]))
    assert not got[0].any() and not got[2].any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_cross_attention_function(t):
    q, k, v = qkv(t, 2, 40, 90, 4, 2, 64)
    g = gen(7)
    a = torch.randint(0, 60, (2, 40), generator=g, device="cuda")
    ranges = torch.stack([a, a + 30], -1).int()
    mask = torch.rand(2, 90, generator=g, device="cuda") < 0.7
    dout = normal(g, *q.shape, t=q.dtype)
    for more in ((-0.3, ranges, mask), (0.5, None, mask), (None, ranges, None)):
        xs = [x.detach().requires_grad_() for x in (q, k, v)]
        out = tokens.cross_attention(*xs, *more)
        ref, lse = tokens.cross_attn_fwd(q, k, v, *more)
        want = tokens.cross_attn_bwd(dout, q, k, v, ref, lse, *more)
        same([out], [ref])
        same(torch.autograd.grad(out, xs, dout), want)
    shared = k.detach()[:1].requires_grad_()  # one sequence's keys for the batch: their gradient is the batch's sum
    out = tokens.cross_attention(q, shared.expand(2, -1, -1, -1), v)
    ref, lse = tokens.cross_attn_fwd(q, shared.expand(2, -1, -1, -1), v)
    want = tokens.cross_attn_bwd(dout, q, shared.expand(2, -1, -1, -1), v, ref, lse)[1]
    same(torch.autograd.grad(out, [shared], dout), [want.sum(0, keepdim=True)])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated8_function(t, act):
    g = gen(9)
    h, dy = normal(g, 3, 5, 600, t=TYPES[t]).requires_grad_(), normal(g, 3, 5, 300, t=TYPES[t])
    y = tokens.gated8(h, act)
    flat = h.detach().view(15, 600)
    ref, codes, bounds = tokens.gate8_fwd(flat[:, :300], flat[:, 300:], act)
    dg, du, _ = tokens.gate8_bwd(dy.view(15, 300), codes, bounds, act)
    assert not torch.equal(dg, du)
    same([y], [ref.view(3, 5, 300)])
    same(torch.autograd.grad(y, [h], dy), [torch.cat([dg, du], 1).view(3, 5, 600)])


def test_gated8_keeps_only_its_codes():
    """Between the passes: two bytes a unit, its bounds, and what the caller keeps itself."""
    x = torch.zeros(1 << 10, 1 << 13, device="cuda", requires_grad=True)
    before = torch.cuda.memory_allocated()
    y = tokens.gated8(x * 1.0)
    kept = torch.cuda.memory_allocated() - before
    units = y.numel()
    assert kept <= 4 * units + 2 * units + 16 * units // 256 + (1 << 16)  # y, codes, bounds
    y.sum().backward()
    assert torch.isfinite(x.grad).all()


@pytest.mark.parametrize("case", [("f32", 2, 40, 100, 2, 2, 64), ("bf16", 2, 40, 100, 2, 2, 64), ("bf16", 2, 1, 4000, 2, 2, 64)], ids=str)
def test_cross_attn_nan_in_a_seen_key_or_value(case):
    """A NaN in a key reaches every row that sees it, in a value its element of theirs; nothing of another head or sequence."""
    q, k, v = qkv(*case)
    k[1, 60, 0, 2] = float("nan")
    v[0, 5, 1, 3] = float("nan")
    n = torch.tensor([[[0, 100]], [[0, 100]]], device="cuda", dtype=torch.int32)
    for ranges in (n, n - torch.tensor([[[0, 90]], [[0, 40]]], device="cuda", dtype=torch.int32)):  # the second: the key is the first past the end
        out, lse = tokens.cross_attn_fwd(q, k, v, ranges=ranges)
        bad, bad_lse = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(lse, dtype=torch.bool)
        bad[0, :, 1, 3] = True
        if ranges is n:
            bad[1, :, 0] = bad_lse[1, 0] = True
        assert torch.equal(out.isnan(), bad) and torch.equal(lse.isnan(), bad_lse)
        dout = normal(gen(2), *q.shape, t=q.dtype)
        dq, dk, dv = tokens.cross_attn_bwd(dout, q, k, v, out, lse, ranges=ranges)
        assert dq[0, :, 1].isnan().all() and torch.isfinite(dq[0, :, 0]).all() and torch.isfinite(dq[1, :, 1]).all()
        assert torch.isfinite(dk[0, :, 0]).all() and torch.isfinite(dv[:, :, 1]).all() and torch.isfinite(dk[1, :, 1]).all()
        past = torch.arange(k.shape[1], device="cuda") >= ranges[:, 0, 1:]
        assert not dk[past].any() and not dv[past].any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_cross_attn_infinities_that_rows_see(t):
    """An infinity in a seen key or value is never lost: bfloat16 has the formula's results, float32 those or NaN, and
    what does not see it is as without it."""
    q, k, v = qkv(t, 2, 40, 100, 2, 2, 64)
    plain, plain_lse = tokens.cross_attn_fwd(q, k, v)
    k2, v2 = k.clone(), v.clone()
    k2[1, 60, 0, 2] = math.inf  # scores of q[..., 2] times infinity: weight 0, or NaN
    v2[0, 5, 1, 3] = math.inf
    out, lse = tokens.cross_attn_fwd(q, k2, v2)
    others = torch.ones_like(out, dtype=torch.bool)
    others[1, :, 0] = others[0, :, 1, 3] = False
    assert torch.equal(out[others], plain[others])
    below, above = q[1, :, 0, 2] < 0, q[1, :, 0, 2] > 0
    assert out[1, above, 0].isnan().all() and lse[1, 0, above].isnan().all()
    hidden = torch.ones(2, 100, dtype=torch.bool, device="cuda")
    hidden[1, 60] = False  # a weight of 0 is a key that is not there
    rest, rest_lse = tokens.cross_attn_fwd(q, k, v, key_mask=hidden)
    gone = out[1, below, 0].isnan().all(-1)
    assert torch.equal(gone, lse[1, 0, below].isnan())
    assert ((out[1, below, 0] - rest[1, below, 0])[~gone].abs() <= (1e-5 if t == "f32" else 0.02)).all()
    assert ((lse[1, 0, below] - rest_lse[1, 0, below])[~gone].abs() <= 1e-5).all()
    if t == "bf16":
        assert not gone.any() and (out[0, :, 1, 3] == math.inf).all()
    else:
        assert (out[0, :, 1, 3].isnan() | (out[0, :, 1, 3] == math.inf)).all()


@pytest.mark.parametrize("way", ["grad", "backward"])
def test_functions_refuse_second_derivatives(way):
    """A gradient's gradient is an error from the GPU's backward threads too; the first comes as without create_graph."""
    q, k, v = (x.requires_grad_() for x in qkv("f32", 1, 6, 20, 2, 2, 32))
    w, cs = torch.ones(32, device="cuda"), torch.ones(20, 16, device="cuda")
    for f in (lambda: tokens.norm_rotate(q, k, w, w, cs, cs)[0], lambda: tokens.cross_attention(q, k, v), lambda: tokens.gated8(q, "gelu")):
        plain, = torch.autograd.grad(f().square().sum() + q.square().sum(), q)
        first, = torch.autograd.grad(f().square().sum() + q.square().sum(), q, create_graph=True)
        assert torch.equal(first.detach(), plain)
        with pytest.raises(RuntimeError, match="differentiated once"):
            torch.autograd.grad(first.square().sum(), q) if way == "grad" else first.square().sum().backward()
