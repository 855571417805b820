"""CPU-side checks of the differentiable functions around the token operators and the rasteriser: the calls that
need the GPU are replaced by plain torch, so that what is tested is the way gradients take."""
import os
import types

import pytest
import torch

from test_tokens_abi import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgsraster.so not built")


@pytest.fixture
def t(monkeypatch):
    """tokens with cubes in the place of the operators: y = x^3, dx = 3 x^2 dy, whatever the shape."""
    from tile_differentiable_rasterizer_amd import tokens

    plain = torch.no_grad()  # the C calls are not recorded
    cube, slope = plain(lambda x: x**3), plain(lambda x, d: 3 * x * x * d)

    def gate_fwd(gate, up, act):
        gate_fwd.last = (gate.clone(), up.clone())
        return gate**3 * up, torch.zeros(2, *gate.shape, dtype=torch.uint8), torch.zeros(1)

    @plain
    def gate_bwd(dy, codes, bounds, act, with_y, dgate, dup):
        gate, up = gate_fwd.last
        dgate.copy_(3 * gate**2 * up * dy)
        dup.copy_(gate**3 * dy)

    monkeypatch.setattr(tokens, "norm_rotate_fwd", lambda q, k, *a: (cube(q), cube(k)))
    monkeypatch.setattr(tokens, "norm_rotate_bwd", lambda dq, dk, q, k, wq, wk, *a: (slope(q, dq), slope(k, dk), torch.zeros_like(wq), torch.zeros_like(wk)))
    monkeypatch.setattr(tokens, "cross_attn_fwd", lambda q, k, v, *a: (cube(q) + cube(k) + cube(v), q.sum()))
    monkeypatch.setattr(tokens, "cross_attn_bwd", lambda d, q, k, v, *a: (slope(q, d), slope(k, d), slope(v, d)))
    monkeypatch.setattr(tokens, "gate8_fwd", gate_fwd)
    monkeypatch.setattr(tokens, "gate8_bwd", gate_bwd)
    return tokens


class Frames:
    """In the place of raster.Rasterizer: an image of the cubes."""

    def __init__(self, means, *rest, **more):
        self.means = means

    def forward(self, cam, with_keys=True):
        return dict(image=self.means**3, grads=None)

    @torch.no_grad()
    def backward(self, fwd, dimage):
        zero = torch.zeros(4, 6)
        return dict(dmeans=3 * self.means**2 * dimage, dscales=zero, dquats=zero, grad_screen=zero, dsh=zero)


def function(t, monkeypatch, which):
    """(an operator of one tensor, the tensor)"""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 4, 2, 8, generator=g).requires_grad_()
    w = torch.ones(8)
    if which == "norm_rotate":
        return (lambda x: t.norm_rotate(x, x, w, w, None, None)[1]), x
    if which == "cross_attention":
        return (lambda x: t.cross_attention(x, x, x)), x
    if which == "gated8":
        return (lambda x: t.gated8(x)), x
    from tile_differentiable_rasterizer_amd import token_decoder

    monkeypatch.setattr(token_decoder.raster, "Rasterizer", Frames)
    rest = [torch.zeros(4, 6) for _ in range(4)]
    return (lambda x: token_decoder.Render.apply(x, *rest, types.SimpleNamespace())), torch.randn(4, 6, generator=g).requires_grad_()


FUNCTIONS = ["norm_rotate", "cross_attention", "gated8", "render"]


@pytest.mark.parametrize("squared", [False, True])
@pytest.mark.parametrize("way", ["grad", "backward"])
@pytest.mark.parametrize("which", FUNCTIONS)
def test_second_derivatives_are_refused(t, monkeypatch, which, way, squared):
    """The backward passes are not differentiable: a gradient's gradient is an error, on whichever path it is asked for and
    with whatever beside it, and never one without the operator's part.  First derivatives come with create_graph too."""
    f, x = function(t, monkeypatch, which)

    def loss():
        y = f(x)
        return (y * y if squared else y).sum() + (x * x).sum()

    plain, = torch.autograd.grad(loss(), x)
    first, = torch.autograd.grad(loss(), x, create_graph=True)
    assert torch.equal(first.detach(), plain)
    with pytest.raises(RuntimeError, match="differentiated once"):
        if way == "grad":
            torch.autograd.grad((first * first).sum(), x)
        else:
            (first * first).sum().backward()


@pytest.mark.parametrize("which", FUNCTIONS)
def test_second_derivatives_of_the_rest_are_not_refused(t, monkeypatch, which):
    """What does not lead through an operator's gradient has its second derivative."""
    f, x = function(t, monkeypatch, which)
    z = torch.ones(3, requires_grad=True)
    gx, gz = torch.autograd.grad(f(x).sum() + (z**3).sum(), (x, z), create_graph=True)
    second, = torch.autograd.grad(gz.sum(), z)
    assert torch.equal(second, 6 * torch.ones(3)) and gx.shape == x.shape


def test_a_frame_is_let_go_with_its_graph(t, monkeypatch):
    """Render keeps its rasteriser and what the frame made until the graph goes, with no cycle for the collector to find."""
    import gc
    import weakref

    f, x = function(t, monkeypatch, "render")
    made = []

    class Kept(Frames):
        def __init__(self, *a, **k):
            super().__init__(*a, **k)
            made.append(weakref.ref(self))

    from tile_differentiable_rasterizer_amd import token_decoder

    monkeypatch.setattr(token_decoder.raster, "Rasterizer", Kept)
    gc.disable()
    try:
        y = f(x)
        (y * y).sum().backward()
        del y
        assert made[0]() is None
        y = f(x)  # and where no backward pass comes
        del y
        assert made[1]() is None
    finally:
        gc.enable()


def test_a_frame_whose_inputs_change_is_refused(t, monkeypatch):
    """The backward pass reads the inputs again: changed in place between the passes they would give another frame's gradients."""
    f, x = function(t, monkeypatch, "render")
    z = x * 1.0
    y = f(z)
    with torch.no_grad():
        z.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_reach_the_calls_on_their_boundaries(dtype):
    """A gradient that is dense but starts off a 16-byte boundary (one of several parts of a cat, say) is copied."""
    from tile_differentiable_rasterizer_amd import tokens

    whole = torch.arange(513.0).to(dtype)
    off = whole[1:].view(1, 2, 4, 64)
    assert off.is_contiguous() and off.data_ptr() % 16
    got = tokens._on_vectors(off)
    assert got.data_ptr() % 16 == 0 and got.is_contiguous() and torch.equal(got, off)
    for taken in (whole[:512].view(1, 2, 4, 64), whole[:512].view(1, 4, 2, 64).transpose(1, 2), whole[:64].expand(1, 2, 4, 64)):
        assert tokens._on_vectors(taken) is taken
    for copied in (whole[:512].view(1, 2, 64, 4).transpose(2, 3), torch.zeros(1, 2, 4, 65, dtype=dtype)[..., 1:], torch.zeros((), dtype=dtype).expand(1, 2, 4, 64)):
        got = tokens._on_vectors(copied)
        assert got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, copied)


class Other:
    """A tensor of another GPU than the current one, and a stand-in for what torch and the library do there."""

    shape, dtype = (1, 2, 4, 64), torch.bfloat16

    def get_device(self):
        return 1


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_tensors_gpu(monkeypatch, current):
    """The tensors' GPU is the current one while a call runs (a launch on a default stream goes to whichever that is), and
    the call gets that GPU's current stream."""
    import contextlib

    from tile_differentiable_rasterizer_amd import tokens

    at = [current]

    @contextlib.contextmanager
    def device(n):
        at.append(n)
        yield
        at.pop()

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda n: 70 + n, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    seen = []
    status = types.SimpleNamespace(value=0)

    def call(*args):
        seen.append((at[-1], args))
        return status.value

    monkeypatch.setattr(tokens, "lib", lambda: types.SimpleNamespace(gs_some_call=call))
    tokens._launch("gs_some_call", Other(), 5, None)
    assert seen == [(1, (5, None, 71))] and at == [current]
    status.value = 1
    with pytest.raises(tokens.raster.GsError, match="gs_some_call"):
        tokens._launch("gs_some_call", Other(), 5, None)
    assert at == [current]


def test_a_stream_of_another_gpu_is_refused():
    """Work would go to the tensors' own GPU's current stream and not to the one that was given."""
    from tile_differentiable_rasterizer_amd import tokens

    def call(*args):
        raise AssertionError("not reached")

    for n in (0, 2):
        with pytest.raises(ValueError, match="stream"):
            tokens._on(types.SimpleNamespace(device_index=n), call, Other())


def test_gated8_shapes(t):
    """Any leading axes, none of them or the last empty; a last axis without two halves is refused, and so is a number."""
    for shape in ((4, 6), (2, 3, 4), (6,), (0, 6), (2, 0, 6), (3, 0), (0, 0)):
        x = torch.ones(shape, requires_grad=True)
        y = t.gated8(x)
        assert y.shape == (*shape[:-1], shape[-1] // 2)
        y.sum().backward()
        assert x.grad.shape == x.shape
    for shape in ((4, 5), (3, 1), (2, 2, 7), ()):
        with pytest.raises(ValueError, match="last axis"):
            t.gated8(torch.ones(shape))
