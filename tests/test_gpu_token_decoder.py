"""The decoder example runs its operators together and learns."""
import pytest
import torch

from tile_differentiable_rasterizer_amd import token_decoder

pytestmark = pytest.mark.gpu


def test_decoder_learns_through_the_rasteriser():
    losses = token_decoder.train(steps=40, size=64, views=2, n_tokens=64, say=None)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.5 * losses[0]


def test_decoder_without_anything_shown():
    """Black images: every state is masked, so the tokens attend to nothing; all gradients stay finite."""
    model = token_decoder.Decoder(27, seed=3)
    out = model(torch.zeros(2, 3, 64, 64, device="cuda"))
    sum(x.square().mean() for x in out).backward()
    assert all(torch.isfinite(x).all() for x in out) and torch.isfinite(model.grad).all()
    assert (model.p["q"].grad == 0).all() and (model.p["kv"].grad == 0).all() and model.p["down"].grad.abs().max() > 0
