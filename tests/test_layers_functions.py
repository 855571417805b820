"""CPU-side checks of layer_norm and group_mm as torch functions: the calls that need the GPU are replaced by plain
torch, so that what is tested is the way gradients take."""
import os

import pytest
import torch

from test_tokens_abi import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgsraster.so not built")


@pytest.fixture
def t(monkeypatch):
    """tokens with cubes in the place of the calls."""
    from tile_differentiable_rasterizer_amd import tokens

    plain = torch.no_grad()  # the C calls are not recorded
    asked = []

    @plain
    def norm_bwd(dy, x, w, eps, with_dw, with_db):
        asked.append((with_dw, with_db))
        return 3 * x * x * dy * w, (x**3 * dy).sum(0) if with_dw else None, dy.sum(0) if with_db else None

    @plain
    def mm_bwd(dy, x, w, offsets, with_dx, with_dw):
        asked.append((with_dx, with_dw))
        return 3 * x * x * (dy @ w[0].t()) if with_dx else None, (x**3).t()[None] @ dy if with_dw else None

    monkeypatch.setattr(tokens, "layer_norm_fwd", plain(lambda x, w, b, eps: x**3 * w + b))
    monkeypatch.setattr(tokens, "layer_norm_bwd", norm_bwd)
    monkeypatch.setattr(tokens, "group_mm_fwd", plain(lambda x, w, offsets: x**3 @ w[0]))
    monkeypatch.setattr(tokens, "group_mm_bwd", mm_bwd)
    tokens_asked = asked
    return tokens, tokens_asked


def function(t, which):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(6, 8, generator=g).requires_grad_()
    w, b, m = torch.randn(8, generator=g), torch.randn(8, generator=g), torch.randn(1, 8, 4, generator=g)
    offsets = torch.tensor([0, 6], dtype=torch.int32)
    return ((lambda a: t.layer_norm(a, w, b)) if which == "layer_norm" else (lambda a: t.group_mm(a, m, offsets))), x


@pytest.mark.parametrize("which", ["layer_norm", "group_mm"])
@pytest.mark.parametrize("through", ["sum", "square"])
def test_second_derivatives_are_refused(t, which, through):
    """Whether the gradient that comes in depends on x as well or not."""
    f, x = function(t[0], which)
    y = f(x)
    first, = torch.autograd.grad(y.sum() if through == "sum" else y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated once"):
        torch.autograd.grad(first.sum(), x)


@pytest.mark.parametrize("which", ["layer_norm", "group_mm"])
def test_a_changed_input_is_an_error(t, which):
    f, x = function(t[0], which)
    a = x * 1
    y = f(a)
    with torch.no_grad():
        a.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_only_what_is_wanted_is_asked_for(t):
    tokens, asked = t
    x, w, b = torch.ones(6, 8, requires_grad=True), torch.ones(8), torch.ones(8, requires_grad=True)
    tokens.layer_norm(x, w, b).sum().backward()
    tokens.group_mm(x.detach(), torch.ones(1, 8, 4, requires_grad=True), torch.tensor([0, 6], dtype=torch.int32)).sum().backward()
    tokens.group_mm(x, torch.ones(1, 8, 4), torch.tensor([0, 6], dtype=torch.int32)).sum().backward()
    assert asked == [(False, True), (False, True), (True, False)] and b.grad.tolist() == [6.0] * 8


def test_leading_axes_and_gradients_that_are_not_dense(t):
    tokens, _ = t
    g = torch.Generator().manual_seed(6)
    x, w, b = torch.randn(2, 3, 8, generator=g).requires_grad_(), torch.randn(8, generator=g), torch.zeros(8)
    for view in (lambda z: z, lambda z: z.transpose(0, 1), lambda z: z[..., None].expand(2, 3, 8, 2)[..., 0]):
        d = torch.randn(2, 3, 8, generator=g) if view(x).shape == x.shape else torch.randn(3, 2, 8, generator=g)
        got, = torch.autograd.grad(tokens.layer_norm(view(x), w, b), x, d)
        want, = torch.autograd.grad(view(x) ** 3 * w, x, d)
        assert torch.allclose(got, want)
    for shape in ((0, 8), (2, 0, 8), (8,), (3, 1, 8)):
        z = torch.ones(shape, requires_grad=True)
        tokens.layer_norm(z, w, b).sum().backward()
        assert z.grad.shape == z.shape


def test_adamw_wants_every_gradient(monkeypatch):
    """A parameter without a gradient is refused before anything is read."""
    from tile_differentiable_rasterizer_amd import tokens

    class State:
        class m:
            is_cuda = True

            @staticmethod
            def get_device():
                return 0

    for grads in ([None], [torch.ones(3), None]):
        with pytest.raises(ValueError, match="gradient for each"):
            tokens.adamw([torch.ones(3)] * len(grads), grads, State, 1e-3, 1)


def test_matrices_that_are_not_dense(t):
    """group_mm takes a matrix whose rows are not dense, as layer_norm does, and still knows when it was changed."""
    tokens, _ = t
    dense = []
    fwd, bwd = tokens.group_mm_fwd, tokens.group_mm_bwd
    tokens.group_mm_fwd = lambda x, *more: dense.append(x.stride(1) == 1) or fwd(x, *more)
    tokens.group_mm_bwd = lambda dy, x, *more: dense.append(x.stride(1) == 1) or bwd(dy, x, *more)
    g = torch.Generator().manual_seed(7)
    w, offsets, d = torch.randn(1, 8, 4, generator=g).double(), torch.tensor([0, 6], dtype=torch.int32), torch.randn(6, 4, generator=g).double()
    for shape, view in (((8, 6), lambda z: z.t()), ((6, 16), lambda z: z[:, ::2]), ((6, 1), lambda z: z.expand(6, 8))):
        z = torch.randn(shape, generator=g).double().requires_grad_()
        got, = torch.autograd.grad(tokens.group_mm(view(z), w, offsets), z, d)
        want, = torch.autograd.grad(view(z) ** 3 @ w[0], z, d)
        assert torch.allclose(got, want)
        x = view(z).detach()
        x = x.clone(memory_format=torch.preserve_format).requires_grad_()
        a = x * 1
        y = tokens.group_mm(a, w, offsets)
        with torch.no_grad():
            a.mul_(2)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    assert dense and all(dense)
    for wrong in (torch.zeros(8), torch.zeros(2, 3, 8)):
        with pytest.raises(ValueError, match="matrices"):
            tokens.group_mm(wrong, w, offsets)


@pytest.fixture
def reached(monkeypatch):
    """tokens on CPU tensors, and the C calls that would be made (their arguments are checked, nothing runs)."""
    from tile_differentiable_rasterizer_amd import tokens

    calls = []
    monkeypatch.setattr(tokens, "_type", lambda t: tokens.TYPES[t.dtype])
    monkeypatch.setattr(tokens, "_launch", lambda name, *args: calls.append(name))
    return tokens, calls


def test_weights_gradients_of_another_number_of_groups_are_refused(reached):
    """Fewer groups than the weights have would be written past their end."""
    tokens, calls = reached
    x, dy, w, offsets = torch.zeros(6, 8), torch.zeros(6, 4), torch.zeros(3, 8, 4), torch.zeros(4, dtype=torch.int32)
    for shape in ((1, 8, 4), (2, 8, 4), (4, 8, 4), (0, 8, 4), (3, 4, 8), (3, 8, 5), (3, 7, 4), (8, 4)):
        with pytest.raises(ValueError):
            tokens.group_mm_bwd(dy, x, w, offsets, dw=torch.zeros(shape))
    assert not calls
    dw = torch.zeros(3, 8, 4)
    assert tokens.group_mm_bwd(dy, x, w, offsets, dw=dw)[1] is dw and calls == ["gs_group_mm_bwd"]


def test_outputs_and_state_of_other_sizes_are_refused(reached):
    """What the other calls write to has the size that they write."""
    tokens, calls = reached
    x, w = torch.zeros(6, 8), torch.zeros(3, 8, 4)
    offsets = torch.zeros(4, dtype=torch.int32)
    for wrong in (torch.zeros(5, 8), torch.zeros(6, 7), torch.zeros(7, 8), torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(8, 6).t()):
        for call in (lambda: tokens.layer_norm_fwd(x, out=wrong), lambda: tokens.layer_norm_bwd(x, x, dx=wrong), lambda: tokens.layer_norm_bwd(wrong, x),
                     lambda: tokens.group_mm_bwd(torch.zeros(6, 4), x, w, offsets, dx=wrong)):
            with pytest.raises(ValueError):
                call()
    for call in (lambda: tokens.group_mm_fwd(x, w, offsets, out=torch.zeros(6, 5)), lambda: tokens.group_mm_fwd(x, w, offsets, out=torch.zeros(5, 4)), lambda: tokens.group_mm_fwd(x, w, offsets[:3]),
                 lambda: tokens.group_mm_fwd(x, w[:, :7], offsets), lambda: tokens.group_mm_bwd(torch.zeros(6, 5), x, w, offsets), lambda: tokens.layer_norm_fwd(x, torch.zeros(7)),
                 lambda: tokens.layer_norm_fwd(x, None, torch.zeros(9)), lambda: tokens.layer_norm_bwd(x, x, torch.zeros(7))):
        with pytest.raises(ValueError):
            call()
    assert not calls
