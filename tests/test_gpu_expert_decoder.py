"""The decoder example with layer norms, experts and AdamW over its tensors: it runs, and its gradients are those of the same
formulas in plain torch."""
import pytest
import torch

from tile_differentiable_rasterizer_amd import token_decoder, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("optimizer", ["adam_q16", "adamw"])
@pytest.mark.parametrize("experts", [0, 1, 4])
def test_decoder_runs(experts, optimizer):
    losses = token_decoder.train(steps=4, size=64, views=2, n_tokens=27, say=None, experts=experts, optimizer=optimizer)
    assert len(losses) == 4 and all(x == x for x in losses)


def test_copies_are_the_parameters():
    model = token_decoder.Decoder(27, experts=3, optimizer="adamw", seed=1)
    before = {k: v.detach().clone() for k, v in model.p.items()}
    sum(x.square().mean() for x in model(torch.rand(2, 3, 64, 64, device="cuda"))).backward()
    model.step(1e-3)
    assert (model.grad == 0).all()
    for k, v in model.p.items():
        assert not torch.equal(v, before[k]) or k == "router", k
        if model.copies[k] is not None:
            assert torch.equal(model.copies[k], v.detach().bfloat16()), k


def test_parameters_that_something_else_changes():
    """The next pass multiplies with what a parameter holds then, whoever wrote it."""
    model, other = (token_decoder.Decoder(27, optimizer="adamw", seed=s) for s in (1, 2))
    images = torch.rand(2, 3, 64, 64, device="cuda")
    for step in range(2):
        want = other(images)
        sum(x.square().mean() for x in model(images)).backward()
        model.step(1e-3)
        with torch.no_grad():
            for k, v in model.p.items():
                v.copy_(other.p[k])
        assert all(torch.equal(a, b) for a, b in zip(model(images), want)), step


def test_feed_forward_against_torch():
    """The expert part of the layer against the same formulas in 64 bits: bfloat16 between the operators and in the results
    (2^-8 each, five on the longest way) and 8-bit codes of the activations (2^-6 of their norm each way)."""
    model = token_decoder.Decoder(75, experts=4, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, 75, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    p = {k: v.detach().bfloat16().requires_grad_() for k, v in model.p.items()}
    d = torch.randn(1, 75, 256, generator=g, device="cuda").bfloat16()
    y = model.feed_forward(x, p)
    got = torch.autograd.grad(y, (x, p["up"], p["down"]), d)
    X, up, down, router = (t.detach().double().requires_grad_() for t in (x, p["up"], p["down"], p["router"]))
    weight, expert = torch.softmax((x[0] @ p["router"]).double(), -1).max(-1)  # the choice is the rounded router's
    rows = []
    soft = torch.softmax(X[0] @ router, -1)
    for i in range(75):
        e = int(expert[i])
        a, b = (X[0, i] @ up[e]).chunk(2)
        rows.append(((torch.nn.functional.silu(a) * b) @ down[e]) * soft[i, e])
    ref = torch.stack(rows)[None]
    want = torch.autograd.grad(ref, (X, up, down), d.double())
    for name, a, b in zip(("y", "x", "up", "down"), (y, *got), (ref.detach(), *want)):
        off = ((a.double() - b).norm() / b.norm()).item()
        assert off <= 5 * 2.0**-8 + 2 * 2.0**-6, (name, off)


def test_router_gradient_against_torch():
    """The router learns through the weight that its softmax gives the chosen expert.  Beside the part's own error (five roundings to
    bfloat16 and the codes, as above) that gradient has the logits' (half a step of up to 4), the products' with the gradient that comes
    in, their sum's, its own as a logit's, and the result's: eight more of 2^-8."""
    model = token_decoder.Decoder(75, experts=4, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, 75, 256, generator=g, device="cuda").bfloat16()
    p = {k: v.detach().bfloat16().requires_grad_() for k, v in model.p.items()}
    d = torch.randn(1, 75, 256, generator=g, device="cuda").bfloat16()
    got, = torch.autograd.grad(model.feed_forward(x, p), p["router"], d)
    X, up, down, router = (t.detach().double() for t in (x[0], p["up"], p["down"], p["router"]))
    router.requires_grad_()
    expert = torch.softmax((x[0] @ p["router"].detach()).double(), -1).argmax(-1)
    soft = torch.softmax(X @ router, -1)
    a, b = torch.matmul(X[:, None], up[expert])[:, 0].chunk(2, -1)
    y = torch.matmul((torch.nn.functional.silu(a) * b)[:, None], down[expert])[:, 0]
    want, = torch.autograd.grad(y * soft.gather(1, expert[:, None]), router, d[0].double())
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= 13 * 2.0**-8 + 2 * 2.0**-6, off


@pytest.mark.parametrize("optimizer", ["adam_q16", "adamw"])
def test_router_moves(optimizer):
    """A step through the whole model changes the router, and its losses are numbers."""
    model = token_decoder.Decoder(64, experts=4, optimizer=optimizer, seed=5)
    before = model.p["router"].detach().clone()
    sum(x.square().mean() for x in model(torch.rand(2, 3, 64, 64, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda"))).backward()
    grad = model.p["router"].grad.clone()
    assert torch.isfinite(grad).all() and (grad != 0).any()
    model.step(1e-3)
    assert torch.isfinite(model.p["router"]).all() and not torch.equal(model.p["router"], before)
    losses = token_decoder.train(steps=8, size=64, views=2, n_tokens=64, say=None, experts=4, optimizer=optimizer)
    assert len(losses) == 8 and all(abs(x) < float("inf") for x in losses)
