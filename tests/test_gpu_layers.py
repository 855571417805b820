"""GPU tests of the operators that train a decoder layer (layer norm, products grouped by rows, AdamW over many tensors)
against plain implementations in 64 bits.

Tolerances follow from what the kernels round, u = 2^-24 (float32) and v = 2^-8 (bfloat16: half a spacing), element by
element from the reference's own sums of absolute values (and 2^-120 for what underflows):

* layer_norm: a sum over a row passes through at most 16 terms in a lane, 6 exchanges and 16 wavefronts: 40 u of its terms.
  So the mean is off by 40 u mean|x|, d = x - mean by that and u |d|, the variance by 2 mean(|d| e_d) + 40 u var; a
  gradient by the same terms through the formula; dw and db by (rows / 256 + 96) u of their terms (a lane's chain of
  rows, then lanes, wavefronts and workgroups).  bfloat16 results are rounded once more.
* group_mm: a sum of K products, (K + 16) u of their absolute sum, and the result's rounding.
* adamw: p is rounded once (u), after a step whose quotient is float32's (4 u of the step); codes are equal but where the
  value lies within 1e-9 of a border between two (the order of float64 operations).
"""
import math

import pytest
import torch

from test_gpu_tokens import TYPES, U, V, close, gen, half_step, normal
from tile_differentiable_rasterizer_amd import raster, tokens

pytestmark = pytest.mark.gpu

# -- layer norm --------------------------------------------------------------------------------


def ln_ref(x, w, b, eps, dy=None):
    """float64 (y, its tolerance) and, with dy, (dx, tolerance, dw, tolerance, db, tolerance)."""
    half, e = half_step(x.dtype), 40 * U
    x = x.double()
    w = torch.ones_like(x[0]) if w is None else w.double()
    b = torch.zeros_like(x[0]) if b is None else b.double()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    d = x - mean(x)
    var = mean(d * d)
    rstd = (var + eps).rsqrt()
    e_d = e * mean(x.abs()) + U * d.abs()
    e_r = 0.5 * (2 * mean(d.abs() * e_d) + mean(e_d * e_d) + e * var) / (var + eps) + 4 * U
    xh = d * rstd
    e_x = rstd * e_d + xh.abs() * (e_r + 2 * U)
    y = xh * w + b
    out = [y, w.abs() * e_x + 3 * U * (xh * w).abs() + 2 * U * b.abs() + half * y.abs()]
    if dy is None:
        return out
    dy = dy.double()
    g = dy * w
    mg, mgx = mean(g), mean(g * xh)
    dx = rstd * (g - mg - xh * mgx)
    e_mg = (e + U) * mean(g.abs())
    e_mgx = mean(g.abs() * e_x) + (e + 4 * U) * mean((g * xh).abs())
    tol = rstd * (e_mg + e_x * mgx.abs() + xh.abs() * e_mgx + 4 * U * (g.abs() + mg.abs() + (xh * mgx).abs())) + (e_r + 2 * U) * dx.abs() + half * dx.abs()
    chain = (x.shape[0] / 256 + 96) * U
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return out + [dx, tol, dw, (dy.abs() * e_x).sum(0) + chain * (dy * xh).abs().sum(0), db, chain * dy.abs().sum(0)]


def ln_check(x, w, b, eps, dy):
    y = tokens.layer_norm_fwd(x, w, b, eps)
    got = tokens.layer_norm_bwd(dy, x, w, eps)
    again = tokens.layer_norm_bwd(dy, x, w, eps)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "the same bits on every call"
    ref = ln_ref(x, w, b, eps, dy)
    for what, value, i in (("y", y, 0), ("dx", got[0], 2), ("dw", got[1], 4), ("db", got[2], 6)):
        close(value, ref[i], ref[i + 1], what)


LN = [(1, 1), (3, 7), (5, 8), (70, 16), (33, 120), (1, 128), (17, 136), (129, 363), (2, 512), (65, 520), (9, 1000), (7, 1024), (300, 1032), (40, 2047),
      (11, 2048), (13, 2056), (6, 4096), (5, 5001), (3, 8192), (4, 8200), (2, 12345), (3, 16384), (4000, 64), (2500, 256), (700, 2048), (1100, 1001)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows, width", LN)
def test_layer_norm(t, rows, width):
    g = gen(rows * 31 + width)
    x = normal(g, rows, width, t=TYPES[t], std=2.0) + 0.5
    ln_check(x, normal(g, width) + 1, normal(g, width), 1e-5, normal(g, rows, width, t=TYPES[t]))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("width", [40, 363, 1536, 5000, 9001])
def test_layer_norm_strides(t, width):
    """Rows of a wider matrix, from any unit on."""
    g, t = gen(width), TYPES[t]
    for off, gap in ((0, 8), (1, 3), (8, 1), (5, 16)):
        wide = normal(g, 50, width + off + gap, t=t)
        x, dy = wide[:, off: off + width], normal(g, 50, width + 1, t=t)[:, 1:]
        ln_check(x, normal(g, width + 1)[1:].clone(), None, 1e-6, dy)
        out = torch.full((50, width + 9), 7.0, dtype=t, device="cuda")
        tokens.layer_norm_fwd(x, out=out[:, 3: 3 + width])
        assert (out[:, :3] == 7).all() and (out[:, 3 + width:] == 7).all()
        assert torch.equal(out[:, 3: 3 + width], tokens.layer_norm_fwd(x))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("width", [24, 700, 1500, 3000, 7000])
def test_layer_norm_in_place(t, width):
    g, t = gen(4), TYPES[t]
    x, dy = normal(g, 30, width, t=t), normal(g, 30, width, t=t)
    w = normal(g, width)
    y, (dx, dw, db) = tokens.layer_norm_fwd(x, w), tokens.layer_norm_bwd(dy, x, w)
    for which in (0, 1):
        a, d = x.clone(), dy.clone()
        got = tokens.layer_norm_bwd(d, a, w, dx=(a, d)[which])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    a = x.clone()
    assert torch.equal(tokens.layer_norm_fwd(a, w, out=a), y)


def test_layer_norm_parts_that_are_not_wanted():
    g = gen(5)
    x, dy, w = normal(g, 900, 300), normal(g, 900, 300), normal(g, 300)
    dx, dw, db = tokens.layer_norm_bwd(dy, x, w)
    for a, b in ((False, True), (True, False), (False, False)):
        got = tokens.layer_norm_bwd(dy, x, w, with_dw=a, with_db=b)
        assert torch.equal(got[0], dx)
        assert torch.equal(got[1], dw) if a else got[1] is None
        assert torch.equal(got[2], db) if b else got[2] is None
    for y in (tokens.layer_norm_fwd(x), tokens.layer_norm_fwd(x, torch.ones(300, device="cuda")), tokens.layer_norm_fwd(x, None, torch.zeros(300, device="cuda"))):
        assert torch.equal(y, tokens.layer_norm_fwd(x))


def test_layer_norm_of_nothing():
    x = torch.zeros(0, 70, device="cuda")
    assert tokens.layer_norm_fwd(x).shape == (0, 70)
    dx, dw, db = tokens.layer_norm_bwd(x, x)
    assert dx.shape == (0, 70) and (dw == 0).all() and (db == 0).all()
    x = torch.zeros(5, 0, device="cuda")
    assert tokens.layer_norm_fwd(x).shape == (5, 0) and tokens.layer_norm_bwd(x, x)[1].shape == (0,)


@pytest.mark.parametrize("t", TYPES)
def test_layer_norm_far_from_zero_and_constant(t):
    """The variance is taken about the mean: rows far from 0 keep their digits; constant rows give b, and a gradient that
    is finite; a NaN or an infinity stays in its row."""
    t, g = TYPES[t], gen(6)
    x = normal(g, 6, 900, t=t)
    x[1] += 1000
    x[2] = 3.0
    x[3] = 0.0
    x[4] *= 1e18  # (squares of 1e36, whose sum is no float32; their mean is one)
    x[5] *= 1e-18
    w, b, dy = normal(g, 900), normal(g, 900), normal(g, 6, 900, t=t)
    ln_check(x, w, b, 1e-5, dy)
    bad = x.clone()
    bad[0, 7], bad[2, 899] = math.nan, math.inf
    y, dx = tokens.layer_norm_fwd(bad, w, b), tokens.layer_norm_bwd(dy, bad, w)[0]
    keep = [1, 3, 4, 5]
    assert torch.equal(y[keep], tokens.layer_norm_fwd(x, w, b)[keep]) and torch.equal(dx[keep], tokens.layer_norm_bwd(dy, x, w)[0][keep])
    assert y[0].isnan().all() and y[2].isnan().all() and dx[0].isnan().all()


def differences(f, x, u, h):
    """The derivative of f at x (float64 of float32 values) along u, by differences of fourth order."""
    at = lambda s: f((x.double() + s * h * u.double()).float()).item()  # noqa: E731
    return (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)


def test_layer_norm_against_differences():
    """float32: what rounding leaves of a difference is 64 u / h of the loss's terms' root sum; h^4 of its fifth derivative, of
    the order of the loss itself (inputs of variance 1)."""
    g = gen(7)
    x, w, b, dy = normal(g, 12, 200), normal(g, 200) + 1, normal(g, 200), normal(g, 12, 200)
    grads = tokens.layer_norm_bwd(dy, x, w, 1e-5)
    for i, at in enumerate((x, w, b)):
        u = normal(g, *at.shape)
        u /= u.norm()
        h = 2.0**-4

        def loss(z):
            a = [x, w, b]
            a[i] = z
            return (tokens.layer_norm_fwd(*a, 1e-5).double() * dy.double()).sum()

        scale = dy.norm().item()
        assert abs((grads[i].double() * u.double()).sum().item() - differences(loss, at, u, h)) <= scale * (h**4 + 64 * U / h), i


@pytest.mark.parametrize("t", TYPES)
def test_layer_norm_function(t):
    """The torch function's gradients are the call's, over leading axes, with expanded and strided gradients."""
    t, g = TYPES[t], gen(8)
    x = normal(g, 3, 5, 130, t=t).requires_grad_()
    w, b = (normal(g, 130) + 1).requires_grad_(), normal(g, 130).requires_grad_()
    y = tokens.layer_norm(x, w, b, 1e-6)
    for dy in (normal(g, 3, 5, 130, t=t), normal(g, 1, 1, 130, t=t).expand(3, 5, 130), normal(g, 3, 130, 5, t=t).transpose(1, 2)):
        got = torch.autograd.grad(y, (x, w, b), dy, retain_graph=True)
        want = tokens.layer_norm_bwd(dy.reshape(15, 130).contiguous(), x.detach().view(15, 130), w.detach(), 1e-6)
        assert torch.equal(got[0].view(15, 130), want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    only, = torch.autograd.grad(tokens.layer_norm(x, w.detach(), None).sum(), x)
    assert only.shape == x.shape
    shared = normal(g, 1, 1, 130, t=t).requires_grad_()  # a row that many share: its gradient is their sum
    tokens.layer_norm(shared.expand(3, 5, 130)).backward(dy)
    one = tokens.layer_norm_bwd(dy.reshape(15, 130).contiguous(), shared.detach().expand(3, 5, 130).reshape(15, 130))[0]
    close(shared.grad.view(130), one.double().sum(0), 16 * half_step(t) * one.double().abs().sum(0), "shared")


def test_layer_norm_far_offsets():
    """Rows whose last units lie past 2^32 bytes and past 2^31 units from the first."""
    width = 1 << 14
    rows = (1 << 31) // width + 3
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    g = gen(9)
    x[-3:] = normal(g, 3, width, t=torch.bfloat16)
    y = tokens.layer_norm_fwd(x)
    assert torch.equal(y[-3:], tokens.layer_norm_fwd(x[-3:].clone())) and (y[:4] == 0).all()
    del y
    dy = torch.zeros_like(x)
    dy[-3:] = normal(g, 3, width, t=torch.bfloat16)
    dx, dw, db = tokens.layer_norm_bwd(dy, x, dx=dy.clone())
    want = tokens.layer_norm_bwd(dy[-3:].clone(), x[-3:].clone())
    assert torch.equal(dx[-3:], want[0])
    close(db, dy[-3:].double().sum(0), 8 * U * dy[-3:].double().abs().sum(0), "db")


# -- products grouped by rows ------------------------------------------------------------------


def offsets_of(sizes, first=0):
    at = [first]
    for n in sizes:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def mm_check(x, w, offsets, dy, what=""):
    """All three products against 64 bits; rows of no group hold what must not count."""
    edge, half = offsets.tolist(), half_step(x.dtype)
    k, n = w.shape[1:]
    y = tokens.group_mm_fwd(x, w, offsets)
    dx, dw = tokens.group_mm_bwd(dy, x, w, offsets)
    again = (tokens.group_mm_fwd(x, w, offsets), *tokens.group_mm_bwd(dy, x, w, offsets))
    assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), again)), "the same bits on every call"
    assert dw.shape == w.shape
    assert (y[: edge[0]] == 0).all() and (y[edge[-1]:] == 0).all() and (dx[: edge[0]] == 0).all() and (dx[edge[-1]:] == 0).all()
    for g, (a, b) in enumerate(zip(edge, edge[1:])):
        X, W, D = x[a:b].double(), w[g].double(), dy[a:b].double()
        for name, got, p, q in (("y", y[a:b], X, W), ("dx", dx[a:b], D, W.t()), ("dw", dw[g], X.t(), D)):
            want = p @ q
            close(got, want, (p.shape[1] + 16) * U * (p.abs() @ q.abs()) + half * want.abs(), f"{what} group {g}: {name}")


def mm_case(t, sizes, k, n, layout="kn", first=0, behind=0, seed=3):
    g, t = gen(seed), TYPES[t]
    rows = first + sum(sizes) + behind
    x, dy = normal(g, rows, k, t=t), normal(g, rows, n, t=t)
    w = normal(g, len(sizes), k, n, t=t) if layout == "kn" else normal(g, len(sizes), n, k, t=t).transpose(1, 2)
    for m in (x, dy):  # rows of no group count for nothing
        m[:first] = math.nan
        m[rows - behind:] = math.inf
    return x, w, offsets_of(sizes, first), dy


MM = [  # sizes, k, n, rows before, rows behind
    ([1], 8, 8, 0, 0), ([1, 0, 2], 1, 1, 0, 0), ([3], 17, 5, 2, 1), ([0, 0, 0], 64, 64, 0, 5), ([64], 64, 64, 0, 0), ([65, 1], 72, 80, 0, 0),
    ([5, 0, 7, 1, 0, 3], 256, 1024, 0, 0), ([128, 129, 127], 128, 128, 1, 2), ([300, 0, 41], 363, 250, 0, 3), ([255, 257, 511], 136, 264, 0, 0),
    ([1000, 30], 512, 328, 0, 40), ([2, 1, 4, 3] * 20, 104, 56, 0, 0), ([700], 1000, 8, 0, 0), ([600], 8, 1000, 0, 0), ([4000], 96, 160, 0, 0),
    ([1, 15, 16, 17, 31, 32, 33], 2048, 520, 0, 0), ([20], 4096, 264, 0, 0), ([700, 900, 500], 768, 640, 0, 0), ([33] * 3, 130, 66, 0, 0), ([50, 3], 65, 129, 0, 0),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("sizes, k, n, first, behind", MM, ids=str)
def test_group_mm(t, sizes, k, n, first, behind, layout):
    mm_check(*mm_case(t, sizes, k, n, layout, first, behind))


@pytest.mark.parametrize("t", TYPES)
def test_group_mm_strides(t):
    """Parts of wider matrices, at 16-byte boundaries and off them; weights of every second group, and one for all."""
    g, T = gen(11), TYPES[t]
    sizes, k, n = [70, 0, 33, 130], 72, 200
    offs = offsets_of(sizes)
    rows = sum(sizes)
    for off in (0, 8, 3):
        x, dy = normal(g, rows, k + 40, t=T)[:, off: off + k], normal(g, rows, n + 24, t=T)[:, off: off + n]
        wide = normal(g, 8, k + 16, n + 16, t=T)
        mm_check(x, wide[::2, off: off + k, off: off + n], offs, dy, f"off {off}")
        mm_check(x, normal(g, 4, n + 8, k + 8, t=T)[:, :n, off: off + k].transpose(1, 2), offs, dy, f"off {off}, transposed")
    x, dy = normal(g, rows, k, t=T), normal(g, rows, n, t=T)
    mm_check(x, normal(g, 1, k, n, t=T).expand(4, k, n), offs, dy, "shared")
    # outputs between what they must not touch
    w = normal(g, 4, k, n, t=T)
    want = (tokens.group_mm_fwd(x, w, offs), *tokens.group_mm_bwd(dy, x, w, offs))
    room = [torch.full(s, 5.0, dtype=T, device="cuda") for s in ((rows + 2, n + 11), (rows + 2, k + 11), (4, k + 2, n + 11), (4, n + 2, k + 11))]
    y, dx, dw, dwt = room[0][1:-1, 3: 3 + n], room[1][1:-1, 3: 3 + k], room[2][:, 1:-1, 3: 3 + n], room[3][:, 1:-1, 3: 3 + k].transpose(1, 2)
    tokens.group_mm_fwd(x, w, offs, out=y)
    tokens.group_mm_bwd(dy, x, w, offs, dx=dx, dw=dw)
    tokens.group_mm_bwd(dy, x, w, offs, with_dx=False, dw=dwt)
    # each is within its own tolerance of the product (alignment chooses the order of a sum), so twice that of the other
    each = torch.repeat_interleave(torch.tensor(sizes, device="cuda"))
    ax, ad, aw = x.double().abs(), dy.double().abs(), w.double().abs()
    for got, ref, terms, mag in ((y, want[0], k, torch.cat([ax[each == i] @ aw[i] for i in range(4)])),
                                 (dx, want[1], n, torch.cat([ad[each == i] @ aw[i].t() for i in range(4)])),
                                 (dw, want[2], rows, ax.t() @ ad), (dwt, want[2], rows, ax.t() @ ad)):
        close(got, ref.double(), 2 * (terms + 16) * U * mag + 3 * half_step(T) * ref.double().abs(), "elsewhere")
    for r, part in zip(room, (y, dx, dw, dwt)):
        part.fill_(5.0)
        assert (r == 5).all()


@pytest.mark.parametrize("t", TYPES)
def test_group_mm_parts_that_are_not_wanted(t):
    x, w, offs, dy = mm_case(t, [50, 20], 64, 96)
    dx, dw = tokens.group_mm_bwd(dy, x, w, offs)
    assert torch.equal(tokens.group_mm_bwd(dy, x, w, offs, with_dw=False)[0], dx) and torch.equal(tokens.group_mm_bwd(dy, x, w, offs, with_dx=False)[1], dw)
    assert tokens.group_mm_bwd(dy, x, w, offs, False, False) == (None, None)


@pytest.mark.parametrize("t", TYPES)
def test_group_mm_of_nothing(t):
    T = TYPES[t]
    e = lambda *s: torch.ones(s, dtype=T, device="cuda")  # noqa: E731
    offs = offsets_of([2, 3])
    assert tokens.group_mm_fwd(e(0, 8), e(2, 8, 8), offsets_of([0, 0])).shape == (0, 8)
    dx, dw = tokens.group_mm_bwd(e(0, 8), e(0, 8), e(2, 8, 8), offsets_of([0, 0]))
    assert dx.shape == (0, 8) and (dw == 0).all()
    y = tokens.group_mm_fwd(e(5, 0), e(2, 0, 8), offs)  # a sum over nothing
    assert y.shape == (5, 8) and (y == 0).all()
    dx, dw = tokens.group_mm_bwd(e(5, 0), e(5, 8), e(2, 8, 0), offs)
    assert (dx == 0).all() and dx.shape == (5, 8) and dw.shape == (2, 8, 0)
    y = tokens.group_mm_fwd(e(5, 8), e(0, 8, 8), offsets_of([]))  # no groups: rows of none
    assert (y == 0).all() and y.shape == (5, 8)


@pytest.mark.parametrize("t", TYPES)
def test_group_mm_offsets_are_cut(t):
    """Offsets outside of [0, rows] count as its ends; what belongs to no group is 0."""
    x, w, _, dy = mm_case(t, [90, 30, 60], 64, 72)
    wild = torch.tensor([-7, 90, 2**31 - 1, 2**31 - 1], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 90, 180, 180], dtype=torch.int32, device="cuda")
    for got, want in zip((tokens.group_mm_fwd(x, w, wild), *tokens.group_mm_bwd(dy, x, w, wild)), (tokens.group_mm_fwd(x, w, tame), *tokens.group_mm_bwd(dy, x, w, tame))):
        assert torch.equal(got, want)
    room = torch.full((182, 72), 3.0, dtype=x.dtype, device="cuda")
    for offs in ([180, 0, 180, 0], [2**31 - 1, -(2**31), 2**31 - 1, 5], [50, 20, 10, 0]):  # what these compute is nobody's, where they write is known
        tokens.group_mm_fwd(x, w, torch.tensor(offs, dtype=torch.int32, device="cuda"), out=room[1:-1])
        tokens.group_mm_bwd(dy, x, w, torch.tensor(offs, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (room[0] == 3).all() and (room[-1] == 3).all()


@pytest.mark.parametrize("t", TYPES)
def test_group_mm_nan_and_infinities_stay_where_they_belong(t):
    """A NaN in a row reaches this row's results and its group's weight gradient, in a weight its group's rows; others keep their bits."""
    x, w, offs, dy = mm_case(t, [40, 25, 70], 80, 48)
    y = tokens.group_mm_fwd(x, w, offs)
    dx, dw = tokens.group_mm_bwd(dy, x, w, offs)
    x[45, 3], w[2, 7, 9], dy[100, 5] = math.nan, math.inf, math.nan
    y2 = tokens.group_mm_fwd(x, w, offs)
    dx2, dw2 = tokens.group_mm_bwd(dy, x, w, offs)
    keep = [i for i in range(65) if i != 45]
    assert torch.equal(y2[keep], y[keep]) and y2[45].isnan().all()
    assert not torch.isfinite(y2[65:, 9]).any() and torch.equal(y2[65:, :9], y[65:, :9])
    assert torch.equal(dx2[:65], dx[:65]) and dx2[100].isnan().all() and not torch.isfinite(dx2[65:, 7]).any()
    assert torch.equal(dw2[0], dw[0]) and dw2[1, 3].isnan().all() and torch.equal(dw2[1, :3], dw[1, :3]) and dw2[2, :, 5].isnan().all() and torch.equal(dw2[2, :, :5], dw[2, :, :5])


def test_group_mm_against_differences():
    """The product is linear in either factor, so one difference is exact but for rounding: 64 u of the terms' root sum."""
    x, w, offs, dy = mm_case("f32", [30, 0, 50], 60, 40)
    dx, dw = tokens.group_mm_bwd(dy, x, w, offs)
    g = gen(12)
    u, z = normal(g, *x.shape), normal(g, *w.shape)
    loss = lambda a, b: (tokens.group_mm_fwd(a, b, offs).double() * dy.double()).sum().item()  # noqa: E731
    scale = math.sqrt(60) * dy.norm().item()
    assert abs((dx.double() * u.double()).sum().item() - (loss(x + u, w) - loss(x - u, w)) / 2) <= 64 * U * scale * 8
    assert abs((dw.double() * z.double()).sum().item() - (loss(x, w + z) - loss(x, w - z)) / 2) <= 64 * U * scale * 8


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("t", TYPES)
def test_group_mm_function(t, layout):
    x, w, offs, dy = mm_case(t, [30, 0, 50], 64, 40, layout)
    a, b = x.clone().requires_grad_(), w.detach().clone(memory_format=torch.preserve_format).requires_grad_()
    y = tokens.group_mm(a, b, offs)
    for d in (dy, dy[:1].expand(80, 40), dy.t().contiguous().t()):
        got = torch.autograd.grad(y, (a, b), d, retain_graph=True)
        want = tokens.group_mm_bwd(d.contiguous(), x, w, offs)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = w[:1].detach().clone().requires_grad_()  # weights that all groups share: their gradients' sum
    tokens.group_mm(x, one.expand(3, 64, 40), offs).backward(dy)
    parts = tokens.group_mm_bwd(dy, x, one.detach().expand(3, 64, 40), offs)[1].double()
    close(one.grad[0], parts.sum(0), 8 * half_step(x.dtype) * parts.abs().sum(0), "shared")
    first, = torch.autograd.grad(tokens.group_mm(a, b, offs).float().square().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated once"):
        torch.autograd.grad(first.float().sum(), a)


def test_group_mm_far_offsets():
    """Rows past 2^31 units from the first, and weights past 2^32 bytes from the first group's."""
    rows, k, n = (1 << 31) // 512 + 300, 512, 64
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    g = gen(13)
    x[-200:] = normal(g, 200, k, t=torch.bfloat16)
    base = torch.zeros((1 << 31) + k * n, dtype=torch.bfloat16, device="cuda")
    w = torch.as_strided(base, (2, k, n), (1 << 31, n, 1))
    w.copy_(normal(g, 2, k, n, t=torch.bfloat16))
    offs = torch.tensor([rows - 200, rows - 100, rows], dtype=torch.int32, device="cuda")
    near = offsets_of([100, 100])
    want = tokens.group_mm_fwd(x[-200:].clone(), w.clone(), near)
    y = tokens.group_mm_fwd(x, w, offs)
    assert torch.equal(y[-200:], want) and (y[:1000] == 0).all()
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    dy[-200:] = normal(g, 200, n, t=torch.bfloat16)
    dx, dw = tokens.group_mm_bwd(dy, x, w, offs)
    nx, nw = tokens.group_mm_bwd(dy[-200:].clone(), x[-200:].clone(), w.clone(), near)
    assert torch.equal(dx[-200:], nx) and torch.equal(dw, nw) and (dx[:1000] == 0).all()


# -- AdamW -------------------------------------------------------------------------------------


def flat_of(state, sizes, values):
    """The units of each tensor of a flat array."""
    out, at = [], 0
    for n in sizes:
        out.append(values[at: at + n])
        at += -(-n // 256) * 256
    return out


def moments_of(state, sizes):
    """float64 moments of each tensor, by the definition of the codes."""
    if state.bounds is None:
        return [x.double() for x in flat_of(state, sizes, state.m)], [x.double() for x in flat_of(state, sizes, state.v)]
    top = state.bounds.double().repeat_interleave(256, 0)
    c, e = state.m.double(), state.v.double()
    return flat_of(state, sizes, top[:, 0] * (c / 127) ** 2 * c.sign()), flat_of(state, sizes, top[:, 1] * (e / 255) ** 4)


def code_check(codes, bound, x, levels, power, floor):
    """codes [n] and bound [blocks] of moments x [n] (float64, one tensor)."""
    pad = -x.numel() % 256
    blocks = torch.nn.functional.pad(x, (0, pad)).view(-1, 256)
    top = blocks.abs().amax(1)
    assert torch.equal(bound, top.float()) or (bound.double() - top).abs().le(2 * U * top).all()
    bound = bound.double()[:, None]
    real = torch.where(bound > 0, (blocks.abs() / torch.where(bound > 0, bound, torch.ones_like(bound))) ** (1 / power) * levels, torch.zeros_like(blocks))
    want = real.round().clamp(max=levels)
    if floor:
        want = torch.where((blocks > 0) & (bound > 0), want.clamp(min=1), want)
    want = (want * blocks.sign()).view(-1)[: x.numel()]
    sure = ((real - real.floor() - 0.5).abs() > 1e-9).view(-1)[: x.numel()]
    assert torch.equal(codes.double()[sure], want[sure]) and (codes.double() - want).abs().max() <= 1


ADAMW = [  # sizes, offset of each tensor in a buffer (so that they are not aligned)
    [1], [7, 300], [256], [255, 257, 1], [1000, 0, 513], [5000, 64, 70_001], [64] * 65, [(i * 37) % 900 for i in range(150)], [300_000, 3]]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("sizes", ADAMW, ids=lambda s: f"{len(s)}_of_{s[0]}")
def test_adamw(sizes, t, bits, off):
    """Three steps, each held to the definition from the state before it."""
    g, T = gen(len(sizes) + bits), TYPES[t]
    views = lambda dt: [torch.zeros(n + 8, dtype=dt, device="cuda")[off: off + n] for n in sizes]  # noqa: E731
    params, copies = views(torch.float32), views(torch.bfloat16)
    for p in params:
        p.copy_(normal(g, p.numel()))
    state, decay = tokens.adamw_state(params, bits), [0.1 * (i % 3) for i in range(len(sizes))]
    lr, b1, b2, eps = 0.01, 0.9, 0.99, 1e-8
    for step in (1, 2, 3):
        grads = views(T)
        for x in grads:
            x.copy_(normal(g, x.numel()) ** 3)
        m, v = moments_of(state, sizes)
        before = [p.double() for p in params]
        tokens.adamw(params, grads, state, lr, step, b1, b2, eps, weight_decay=decay, copies=copies)
        top, at = state.bounds, 0
        mc, vc = flat_of(state, sizes, state.m), flat_of(state, sizes, state.v)
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            gd = grads[i].double()
            mi, vi = b1 * m[i] + (1 - b1) * gd, b2 * v[i] + (1 - b2) * gd * gd
            move = lr * (mi / (1 - b1**step)) / ((vi / (1 - b2**step)).sqrt() + eps)
            want = before[i] * (1 - lr * decay[i]) - move
            close(params[i], want, U * want.abs() + 4 * U * move.abs(), f"tensor {i}")
            assert torch.equal(copies[i], params[i].bfloat16())
            if bits == 32:
                # a sum of two float64 products that cancel: each of three operations here and there is 2^-53 of the terms off
                close(mc[i], mi, 2 * U * mi.abs() + 6 * 2.0**-53 * (b1 * m[i].abs() + (1 - b1) * gd.abs()), "m")
                close(vc[i], vi, 2 * U * vi.abs(), "v")
            else:
                nb = -(-n // 256)
                code_check(mc[i], top[at: at + nb, 0], mi, 127, 2, False)
                code_check(vc[i], top[at: at + nb, 1], vi, 255, 4, True)
                at += nb
    behind = torch.ones_like(state.m, dtype=torch.bool)
    for x in flat_of(state, sizes, behind):
        x.fill_(False)
    assert (state.m[behind] == 0).all() and (state.v[behind] == 0).all(), "behind a tensor's last unit"
    dm, dv = tokens.adamw_moments(state)
    m, v = moments_of(state, sizes)
    for i in range(len(sizes)):
        close(flat_of(state, sizes, dm)[i], m[i], 2 * U * m[i].abs(), "m")
        close(flat_of(state, sizes, dv)[i], v[i], 2 * U * v[i].abs(), "v")


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_units_far_apart(bits):
    """A block whose gradients span thirty orders of magnitude: no step is larger than a bias-corrected one can be
    (|m| / sqrt(v) of 1 and what the codes' spacing adds), and a unit without gradients does not move."""
    n = 256
    grads = [torch.logspace(-30, 0, n, device="cuda") * torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0)]
    grads[0][5] = 0.0
    params = [torch.zeros(n, device="cuda")]
    state = tokens.adamw_state(params, bits)
    for step in range(1, 30):
        before = params[0].clone()
        tokens.adamw(params, grads, state, 1e-3, step, eps=1e-12)
        assert torch.isfinite(params[0]).all()
        # m stands at most half a code above what it is (3/2 squared) and v's root at most as far below
        assert (params[0] - before).abs().max() <= 1e-3 * 5.1
    assert params[0][5] == 0


def test_adamw_grad_scale_and_single_decay():
    g = gen(21)
    p = [normal(g, 700), normal(g, 90)]
    q = [x.clone() for x in p]
    grads = [normal(g, 700), normal(g, 90)]
    a, b = tokens.adamw_state(p), tokens.adamw_state(q)
    scale = torch.tensor([0.25], device="cuda")
    tokens.adamw(p, grads, a, 1e-2, 1, weight_decay=0.3, grad_scale=scale)
    tokens.adamw(q, [x * 0.25 for x in grads], b, 1e-2, 1, weight_decay=[0.3, 0.3])
    assert all(torch.equal(x, y) for x, y in zip(p + [a.m, a.v, a.bounds], q + [b.m, b.v, b.bounds]))


@pytest.mark.parametrize("bad", [math.nan, math.inf, 1e25])
def test_adamw_keeps_what_is_not_finite_in_its_block(bad):
    """8 bits: a moment that is no float32 makes its block's bound NaN (codes 0); other blocks keep their bits."""
    g = gen(22)
    start, grad = normal(g, 1024), normal(g, 1024)
    runs = []
    for x in (None, bad):
        p, gr = start.clone(), grad.clone()
        if x is not None:
            gr[300] = x
        state = tokens.adamw_state([p])
        tokens.adamw([p], [gr], state, 1e-3, 1)
        runs.append((p, state))
    (p, a), (q, b) = runs
    others = torch.arange(1024, device="cuda") != 300
    assert torch.equal(p[others], q[others])  # this step's parameters come from the moments before they are codes
    assert b.bounds[1, 1].isnan() and (b.v[256:512] == 0).all()
    assert torch.equal(a.m[512:], b.m[512:]) and torch.equal(a.bounds[[0, 2, 3]], b.bounds[[0, 2, 3]])


def test_adamw_marks_its_tensors_as_changed():
    """A backward pass that needs a parameter as it was is an error."""
    p = normal(gen(23), 50).requires_grad_()
    y = (p * p).sum()
    tokens.adamw([p], [torch.ones(50, device="cuda")], tokens.adamw_state([p]), 1e-3, 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_adamw_refuses():
    p, g = [torch.zeros(300, device="cuda")], [torch.zeros(300, device="cuda")]
    state = tokens.adamw_state(p)
    go = lambda p=p, g=g, s=state, lr=1e-3, step=1, **more: tokens.adamw(p, g, s, lr, step, **more)  # noqa: E731
    go()
    half = [x.bfloat16() for x in p]
    for bad in (dict(g=g * 2), dict(p=half), dict(g=[g[0][:200]]), dict(p=[torch.zeros(600, device="cuda")[::2]]), dict(g=[g[0].half()]), dict(s=tokens.adamw_state(p * 3)),
                dict(p=p * 2, g=g * 2, s=tokens.adamw_state(p * 2)), dict(copies=[p[0]]), dict(copies=half * 2), dict(weight_decay=[0.1, 0.2]), dict(g=[g[0].cpu()]),
                dict(grad_scale=torch.ones(2, device="cuda")), dict(grad_scale=torch.ones(1)), dict(s=tokens.AdamWState(state.m, state.v)),
                dict(s=tokens.AdamWState(state.m.view(torch.uint8), state.v, state.bounds))):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=math.nan), dict(weight_decay=math.inf)):
        with pytest.raises(raster.GsError):
            go(**bad)


# -- together ----------------------------------------------------------------------------------


def make_layer(g, T, width=96, hidden=160, experts=3):
    w = dict(norm=normal(g, width) * 0.1 + 1, bias=normal(g, width) * 0.1, up=normal(g, experts, width, 2 * hidden, std=width**-0.5),
             down=normal(g, experts, hidden, width, std=hidden**-0.5))
    return w, [w["norm"], w["bias"], w["up"], w["down"]]


def layer_step(x, dy, w, copies, offs):
    """Norm, experts with a gated activation between, and the gradients of everything, by the raw calls."""
    h = tokens.layer_norm_fwd(x, w["norm"], w["bias"])
    a = tokens.group_mm_fwd(h, copies[0], offs)
    half = a.shape[1] // 2
    y, codes, bounds = tokens.gate8_fwd(a[:, :half], a[:, half:])
    out = tokens.group_mm_fwd(y, copies[1], offs)
    d_y, d_down = tokens.group_mm_bwd(dy, y, copies[1], offs)
    d_a = torch.empty_like(a)
    tokens.gate8_bwd(d_y, codes, bounds, with_y=False, dgate=d_a[:, :half], dup=d_a[:, half:])
    d_h, d_up = tokens.group_mm_bwd(d_a, h, copies[0], offs)
    dx, d_norm, d_bias = tokens.layer_norm_bwd(d_h, x, w["norm"])
    return out, dx, [d_norm, d_bias, d_up, d_down]


def train_step(x, dy, w, params, copies, states, offs, step):
    out, dx, grads = layer_step(x, dy, w, copies, offs)
    tokens.adamw(params[:2], grads[:2], states[0], 1e-3, step)  # float32 gradients
    tokens.adamw(params[2:], grads[2:], states[1], 1e-3, step, weight_decay=0.01, copies=copies)
    return [out, dx, *grads]


def layer_setup(seed=31):
    g, T = gen(seed), torch.bfloat16
    w, params = make_layer(g, T)
    copies = [p.to(T) for p in params[2:]]
    states = tokens.adamw_state(params[:2], 32), tokens.adamw_state(params[2:], 8)
    x, dy, offs = normal(g, 75, 96, t=T), normal(g, 75, 96, t=T, std=0.1), offsets_of([40, 0, 30], 2)
    return x, dy, w, params, copies, states, offs


def everything(params, copies, states):
    return [x.clone() for x in (*params, *copies, *[t for s in states for t in (s.m, s.v, *([] if s.bounds is None else [s.bounds]))])]


def test_layer_trains_as_its_formulas_say():
    """One layer's pass by the raw calls against torch's gradients in 64 bits of the same formulas; bfloat16 activations
    between the operators round to v each, four of them on the longest way: 8 v of the gradients' norms."""
    x, dy, w, params, copies, states, offs = layer_setup()
    out, dx, grads = layer_step(x, dy, w, copies, offs)
    leaf = [t.double().requires_grad_() for t in (x, w["norm"], w["bias"], *copies)]
    X, n, b, up, down = leaf
    h = torch.nn.functional.layer_norm(X, (96,), n, b, 1e-5)
    edge = offs.tolist()
    ref = torch.zeros(75, 96, dtype=torch.float64, device="cuda")
    for e in range(3):
        a, z = (h[edge[e]: edge[e + 1]] @ up[e]).chunk(2, -1)
        ref[edge[e]: edge[e + 1]] = (torch.nn.functional.silu(a) * z) @ down[e]
    want = torch.autograd.grad(ref, leaf, dy.double())
    # gate8's codes: 1/510 of a block's span, of the activations' norm at most 2^-6 each way
    for name, got, r in (("out", out, ref.detach()), ("dx", dx, want[0]), *zip(("norm", "bias", "up", "down"), grads, want[1:])):
        off = (got.double() - r).norm() / r.norm()
        assert off <= 8 * V + 2.0**-5, (name, off.item())


def test_layer_on_other_streams_at_once():
    """Two layers step on streams of their own, beside each other: the same bits as one after another."""
    sets = [layer_setup(31), layer_setup(32)]
    want = []
    for s in [layer_setup(31), layer_setup(32)]:
        got = [train_step(*s, step) for step in range(1, 4)]
        want.append([*(x.clone() for y in got for x in y), *everything(*s[3:6])])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for step in range(1, 4):
        for i, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i] += train_step(*s, step)
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        assert all(torch.equal(a, b) for a, b in zip(got[i] + everything(*s[3:6]), want[i])), i


def test_layer_stream_argument():
    """Work on a stream given by argument while the current one allocates and overwrites."""
    side = torch.cuda.Stream()
    x, dy, w, params, copies, states, offs = layer_setup()

    def step(stream):
        h = tokens.layer_norm_fwd(x, w["norm"], w["bias"], stream=stream)
        a = tokens.group_mm_fwd(h, copies[0], offs, stream=stream)
        d_h, d_up = tokens.group_mm_bwd(a, h, copies[0], offs, stream=stream)
        dx, dn, db = tokens.layer_norm_bwd(d_h, x, w["norm"], stream=stream)
        p, s = params[2].clone(), tokens.adamw_state([params[2]])
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        tokens.adamw([p], [d_up], s, 1e-3, 1, stream=stream)
        return [h, a, d_h, d_up, dx, dn, db, p, *tokens.adamw_moments(s, stream=stream)]

    want = step(None)
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk


def test_layer_in_a_graph():
    """A captured training step replays to the eager results, with other work between the replays (lr and step are the
    captured call's)."""
    x, dy, w, params, copies, states, offs = layer_setup()
    twin = layer_setup()
    train_step(*layer_setup(), 5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train_step(x, dy, w, params, copies, states, offs, 5)
    for i in range(4):
        new, sizes = normal(gen(60 + i), *x.shape, t=x.dtype), [[40, 0, 30], [0, 75, 0], [25, 25, 25], [1, 2, 3]][i]
        for s in ((x, offs), (twin[0], twin[6])):
            s[0].copy_(new)
            s[1].copy_(offsets_of(sizes))
        want = [t.clone() for t in train_step(*twin, 5)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert all(torch.equal(a, b) for a, b in zip(everything(params, copies, states), everything(*twin[3:6]))), i


def test_two_graphs_on_one_workspace():
    """Graphs that share a workspace replay one after another to the eager results."""
    g = gen(41)
    x, dy = normal(g, 900, 512), normal(g, 900, 512)
    ws = torch.empty(tokens.lib().gs_layer_norm_workspace_bytes(900, 512), dtype=torch.uint8, device="cuda")
    graphs, got, want = [], [], []
    for i in range(2):
        want.append([t.clone() for t in tokens.layer_norm_bwd(dy * (i + 1), x, workspace=ws)])
    torch.cuda.synchronize()
    scaled = [dy * 1, dy * 2]
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(tokens.layer_norm_bwd(scaled[i], x, workspace=ws))
        graphs.append(graph)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_functions_in_a_graph():
    """Forward and gradients of the torch functions captured together, replayed with eager work between."""
    x, dy, w, params, copies, states, offs = layer_setup(33)
    leaf = [t.detach().clone().requires_grad_() for t in (x, w["norm"], w["bias"], copies[0])]

    def run():
        a, n, b, up = leaf
        y = tokens.group_mm(tokens.layer_norm(a, n, b), up, offs)
        return [y.detach(), *torch.autograd.grad(y, leaf, dy.new_ones(y.shape))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(3):
        with torch.no_grad():
            leaf[0].copy_(normal(gen(70 + i), *x.shape, t=x.dtype))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("order", [(1, 0, 2), (2, 0, 1), (1, 2, 0), (0, 2, 1), (2, 1, 0)])
def test_group_mm_weights_in_any_order(t, order):
    """Axes of the weights in any order in memory, so long as one of the last two is dense; gradients lie as they do."""
    x, w, offs, dy = mm_case(t, [30, 0, 50], 64, 40)
    lies = w.permute(order).contiguous().permute([order.index(i) for i in range(3)])
    assert torch.equal(lies, w)
    if 1 not in lies.stride()[1:]:
        with pytest.raises(ValueError, match="dense"):
            tokens.group_mm_fwd(x, lies, offs)
        return
    mm_check(x, lies, offs, dy, str(order))
    assert tokens.group_mm_bwd(dy, x, lies, offs)[1].stride() == lies.stride()
