"""CPU-side checks of the calls that train a decoder layer (layer norm, products grouped by rows, AdamW): bad arguments
are refused before any HIP call, workspaces are sized, the binding refuses what the C calls cannot see."""
import ctypes as C
import math
import os

import pytest

from test_tokens_abi import A, BAD, LIB, OK, OVERFLOW, WORKSPACE, tokens

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgsraster.so not built")


def layer_norm_call(rows=3, width=64, type=0, eps=1e-5, x=A, stride=64, w=A, b=A, y=A, y_stride=64, bwd=False, dw=A, db=A, dy=A, dy_stride=64, ws=A, ws_bytes=1 << 30):
    L = tokens().lib()
    if bwd:
        return L.gs_layer_norm_bwd(rows, width, type, eps, dy, dy_stride, x, stride, w, y, y_stride, dw, db, ws, ws_bytes, None)
    return L.gs_layer_norm_fwd(rows, width, type, eps, x, stride, w, b, y, y_stride, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=A + 1), dict(type=1, x=A + 2), dict(y=None), dict(y=A + 1), dict(y_stride=63), dict(y_stride=0), dict(stride=-64),
                                 dict(w=A + 2), dict(type=2), dict(type=-1), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(rows=-1), dict(width=-1)], ids=str)
@pytest.mark.parametrize("bwd", [False, True])
def test_layer_norm_refuses(bad, bwd):
    assert layer_norm_call(bwd=bwd, **bad) == BAD


def test_layer_norm_limits():
    for bwd in (False, True):
        assert layer_norm_call(rows=1 << 31, bwd=bwd) == OVERFLOW
        assert layer_norm_call(width=16385, stride=16385, y_stride=16385, dy_stride=16385, bwd=bwd) == OVERFLOW
        assert layer_norm_call(width=1 << 62, bwd=bwd) == OVERFLOW
        assert layer_norm_call(width=0, x=None, y=None, dy=None, bwd=bwd) == OK
    assert layer_norm_call(b=A + 2) == BAD
    assert layer_norm_call(rows=0, x=None, y=None) == OK
    assert layer_norm_call(rows=0, x=None, y=None, dy=None, dw=None, db=None, ws=None, bwd=True) == OK
    for bad in (dict(dy=None), dict(dy=A + 1), dict(dy_stride=-1), dict(dw=A + 1), dict(db=A + 2)):
        assert layer_norm_call(bwd=True, **bad) == BAD
    many = dict(bwd=True, rows=5000)
    for short in (dict(ws=None), dict(ws=A + 8), dict(ws_bytes=100)):
        assert layer_norm_call(**many, **short) == WORKSPACE
    size = tokens().lib().gs_layer_norm_workspace_bytes
    assert 0 < size(5000, 64) < 1 << 22 and size(0, 64) == 0 and size(5000, 0) == 0 and size(-1, 64) == 0 and size(5, 1 << 20) == 0
    assert size(5000, 16384) <= 1 << 28


def group_call(x=A, xs=None, w=A, w_strides=None, y=A, ys=None, bwd=False, dw=A, dw_strides=None, dx=A, dxs=None, ws=A, ws_bytes=1 << 40, **change):
    t = tokens()
    s = dict(rows=20, k=64, n=96, groups=3, type=0, offsets=A)
    s.update(change)
    p, k, n = t.GsGroupMM(**s), s["k"], s["n"]
    strides = w_strides or (k * n, n, 1)
    W = t.GsWeights(w, *strides)
    xs, ys = k if xs is None else xs, n if ys is None else ys
    if bwd:
        return t.lib().gs_group_mm_bwd(p, y, ys, x, xs, W, dx, k if dxs is None else dxs, t.GsWeights(dw, *(dw_strides or strides)), ws, ws_bytes, None)
    return t.lib().gs_group_mm_fwd(p, x, xs, W, y, ys, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=A + 1), dict(type=1, x=A + 2), dict(xs=-64), dict(w=None), dict(w=A + 1), dict(w_strides=(6144, 95, 1)), dict(w_strides=(6144, 2, 2)),
                                 dict(w_strides=(6144, 1, 63)), dict(w_strides=(-1, 96, 1)), dict(w_strides=(6144, 96, -1)), dict(y=None), dict(y=A + 1), dict(ys=-1), dict(type=2), dict(rows=-1),
                                 dict(k=-1), dict(n=-1), dict(groups=-1), dict(offsets=None), dict(offsets=A + 2)], ids=str)
@pytest.mark.parametrize("bwd", [False, True])
def test_group_mm_refuses(bad, bwd):
    assert group_call(bwd=bwd, **bad) == BAD


def test_group_mm_limits():
    for bwd in (False, True):
        for big in (dict(rows=1 << 31), dict(k=1 << 25), dict(n=1 << 25), dict(groups=65537), dict(rows=1 << 30, k=1 << 20, n=1 << 20)):
            assert group_call(bwd=bwd, **big) == OVERFLOW, big
    assert group_call(ys=95) == BAD and group_call(ys=0) == BAD
    for bad in (dict(dxs=63), dict(dxs=0), dict(dx=A + 1), dict(dw=A + 1), dict(dw_strides=(6143, 96, 1)), dict(dw_strides=(0, 96, 1)), dict(dw_strides=(6144, 0, 1)), dict(dw_strides=(6144, 2, 2))):
        assert group_call(bwd=True, **bad) == BAD, bad
    assert group_call(rows=0, x=None, y=None, w=None) == OK
    assert group_call(n=0, y=None, w=None) == OK
    assert group_call(bwd=True, dx=None, dw=None, y=None, x=None, w=None) == OK  # nothing is wanted
    t = tokens()
    assert t.lib().gs_group_mm_fwd_workspace_bytes(None) == 0 and t.lib().gs_group_mm_bwd_workspace_bytes(None) == 0


def adamw_call(n=(300, 0, 5), param=A, grad=A, copy=None, decay=0.0, grad_type=0, bits=8, m=A, v=A, bounds=A, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, scale=None, count=None):
    t = tokens()
    table = (t.GsAdamWTensor * max(1, len(n)))(*[t.GsAdamWTensor(param, grad, copy, x, decay) for x in n])
    return t.lib().gs_adamw(len(n) if count is None else count, table, grad_type, bits, m, v, bounds, t.GsAdamWParams(lr, beta1, beta2, eps, step), scale, None)


@pytest.mark.parametrize("bad", [dict(param=None), dict(param=A + 2), dict(grad=None), dict(grad=A + 1), dict(grad_type=1, grad=A + 2), dict(copy=A + 1), dict(n=(300, -1)), dict(decay=math.nan),
                                 dict(grad_type=2), dict(bits=16), dict(bits=0), dict(m=None), dict(m=A + 8), dict(v=None), dict(v=A + 8), dict(bounds=None), dict(bounds=A + 4),
                                 dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-9), dict(eps=math.inf), dict(step=0), dict(scale=A + 1),
                                 dict(count=-1)], ids=str)
def test_adamw_refuses(bad):
    assert adamw_call(**bad) == BAD


def test_adamw_limits():
    assert adamw_call(n=(1 << 35,)) == OVERFLOW
    assert adamw_call(n=(1 << 34, 1 << 34)) == OVERFLOW
    assert adamw_call(n=(1 << 62,)) == OVERFLOW
    assert adamw_call(n=(), m=None, v=None, bounds=None) == OK
    assert adamw_call(n=(0, 0), param=None, grad=None, m=None, v=None, bounds=None) == OK
    t = tokens()
    assert t.lib().gs_adamw(1, None, 0, 8, A, A, A, t.GsAdamWParams(1e-3, 0.9, 0.999, 1e-8, 1), None, None) == BAD
    assert t.lib().gs_adamw(0, None, 0, 8, A, A, A, None, None, None) == BAD
    M = t.lib().gs_adamw_moments
    assert M(0, None, None, None, None, None, None) == OK and M(-1, A, A, A, A, A, None) == BAD and M(1 << 27, A, A, A, A, A, None) == OVERFLOW
    for i in range(5):
        args = [A] * 5
        for wrong in (None, A + 4):
            args[i] = wrong
            assert M(3, *args, None) == BAD


def test_structures_are_the_headers():
    t = tokens()
    assert C.sizeof(t.GsAdamWTensor) == 40 and C.sizeof(t.GsAdamWParams) == 40 and C.sizeof(t.GsGroupMM) == 40 and C.sizeof(t.GsWeights) == 32


def test_binding_refuses_what_the_c_calls_cannot_see():
    import torch

    t = tokens()
    x, w, offs = torch.zeros(4, 8), torch.zeros(2, 8, 8), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: t.layer_norm_fwd(x), lambda: t.layer_norm_fwd(torch.zeros(4, 8, dtype=torch.float16)), lambda: t.layer_norm_fwd(torch.zeros(4)),
                 lambda: t.layer_norm_bwd(x, x), lambda: t.layer_norm(torch.zeros(())), lambda: t.group_mm_fwd(x, w, offs), lambda: t.group_mm_bwd(x, x, w, offs),
                 lambda: t.group_mm_fwd(x[0], w, offs), lambda: t.adamw_state([]), lambda: t.adamw_state([x], bits=16),
                 lambda: t.adamw([x], [x], t.adamw_state([x]), 1e-3, 1), lambda: t.adamw([x], [], t.adamw_state([x]), 1e-3, 1), lambda: t.adamw_moments(t.adamw_state([x]))):
        with pytest.raises(ValueError):
            call()


def test_moments_in_32_bits_are_the_states_own():
    import torch

    t = tokens()
    s = t.adamw_state([torch.zeros(300), torch.zeros(0), torch.zeros(5)], bits=32)
    assert s.m.shape == (768,) and t.adamw_moments(s)[0] is s.m


def moments_call(blocks):
    return tokens().lib().gs_adamw_moments(blocks, A, A, A, A, A, None)


def test_weights_gradients_that_lie_between_each_other():
    """[k][groups][n] and [n][groups][k] are taken as an output; a row that starts inside of another's is not."""
    for strides, ok in (((96, 288, 1), True), ((96, 287, 1), False), ((95, 288, 1), False), ((64, 1, 192), True), ((64, 1, 191), False), ((63, 1, 192), False), ((6144, 96, 1), True)):
        how = dict(bwd=True, dx=None, dw_strides=strides)
        assert (group_call(rows=0, x=None, y=None, w=None, ws=None, **how) != BAD) == ok, strides
