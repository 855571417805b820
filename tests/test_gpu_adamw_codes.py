"""AdamW's 8-bit codes where a block's bound is close to the smallest float32s, against 64 bits.

There a bound lies up to half a spacing (2^-150) from its block's largest moment, which is a large part of it: the ratio of the
two passes 1 by as much, and codes stay at their largest, 127 and 255.  Codes are compared with the definition's for the bound that
the call left: equal, but where the value lies within 1e-9 of a border between two (the order of float64 operations)."""
import pytest
import torch

from tile_differentiable_rasterizer_amd import tokens

pytestmark = pytest.mark.gpu

LEAST = 2.0**-149  # float32's spacing below 2^-126
B1, B2 = 0.9, 0.999


def decoded(state):
    """float64 moments [blocks][256] on the host, by the definition of the codes."""
    m, v, top = state.m.cpu().double().view(-1, 256), state.v.cpu().double().view(-1, 256), state.bounds.cpu().double()
    return top[:, :1] * (m / 127) ** 2 * m.sign(), top[:, 1:] * (v / 255) ** 4


def codes_held(codes, bound, x, levels, power, floor):
    """codes and bound [blocks] that a call left of moments x [blocks][256]."""
    codes, bound = codes.cpu().double().view(-1, 256), bound.cpu().double()
    top = x.abs().amax(1)
    half = 0.5 * torch.maximum(top.log2().floor().exp2() * 2.0**-23, torch.full_like(top, LEAST))  # half a spacing
    # and 2^-53 of the moment for each of the eight operations, here and there, that it comes from: a tenth of the bounds lies halfway
    off = int(((bound - top).abs() > half + 8 * 2.0**-53 * top).sum())
    assert off == 0, "bounds are the largest moments, rounded"
    some = bound[:, None] > 0
    real = torch.where(some, (x.abs() / torch.where(some, bound[:, None], 1.0)) ** (1 / power) * levels, 0.0)
    want = real.round().clamp(max=levels)
    if floor:
        want = torch.where((x > 0) & some, want.clamp(min=1), want)
    want = want * x.sign()
    sure = ((real - real.floor() - 0.5).abs() > 1e-9) | (real > levels)
    assert torch.equal(codes[sure], want[sure]), f"{int((codes != want)[sure].sum())} codes, first {codes[sure][codes[sure] != want[sure]][:4].tolist()}"
    assert (codes - want).abs().max() <= 1


def one_step(state, grad):
    """A step on one tensor, held to the definition from the state before it."""
    m, v = decoded(state)
    g = grad.cpu().double().view(-1, 256)
    tokens.adamw([torch.zeros(grad.shape, device="cuda")], [grad], state, 1e-3, 7, B1, B2)
    codes_held(state.m, state.bounds[:, 0], B1 * m + (1 - B1) * g, 127, 2, False)
    codes_held(state.v, state.bounds[:, 1], B2 * v + (1 - B2) * g * g, 255, 4, True)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_small_gradients(t):
    """Second moments from 2^-149 and below up to 2^-126: blocks of gradients from 1e-23 to 1e-17, all alike or of all sizes below."""
    g = torch.Generator().manual_seed(1)
    size = torch.logspace(-23, -17, 601)[:, None]
    for x in (size.expand(601, 256), size * torch.rand(601, 256, generator=g), size * torch.randn(601, 256, generator=g) ** 3):
        grad = x.contiguous().to("cuda", t).view(-1)
        state = tokens.adamw_state([grad])
        for _ in range(3):
            one_step(state, grad)


@pytest.mark.parametrize("which", [0, 1])
def test_small_bounds(which):
    """A step without gradients from blocks with bounds of 1 to 400 times 2^-149, and random codes."""
    g = torch.Generator().manual_seed(2)
    n = 400
    grad = torch.zeros(n * 256, device="cuda")
    state = tokens.adamw_state([grad])
    for full in (False, True):
        state.m.copy_(torch.randint(-127, 128, (n * 256,), generator=g))
        state.v.copy_(torch.randint(1, 256, (n * 256,), generator=g))
        if full:
            state.m.fill_(-127)
            state.v.fill_(255)
        state.bounds.fill_(1e-3)
        state.bounds[:, which] = (torch.arange(1, n + 1, dtype=torch.float64) * LEAST).float().cuda()
        one_step(state, grad)


def test_moments_that_die_out_keep_their_signs():
    """Units without gradients for as long as their first moments take to pass through all of float32's sizes."""
    g = torch.Generator(device="cuda").manual_seed(3)
    p, grad = torch.zeros(2048, device="cuda"), torch.randn(2048, generator=g, device="cuda") * 1e-4
    state = tokens.adamw_state([p])
    tokens.adamw([p], [grad], state, 1e-3, 1)
    sign, zero = state.m.sign(), torch.zeros_like(grad)
    for step in range(2, 1001):
        tokens.adamw([p], [zero], state, 1e-3, step)
        if step > 700:
            assert (state.m.sign() * sign >= 0).all(), step


@pytest.mark.parametrize("beta2, last", [(0.999, 255), (0.99, 199), (0.95, 39)])
def test_codes_that_stay(beta2, last):
    """What the header says of a run: beside a unit that holds the bounds, codes without gradients fall to 0.5 / (1 - beta^(1 / power)) and
    stay there; without that unit's gradient the block decays as a whole, its codes unchanged."""
    assert int(0.5 / (1 - 0.9**0.5)) == 9 and min(int(0.5 / (1 - beta2**0.25)), 255) == last
    p, grad = torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
    state = tokens.adamw_state([p])
    m = (torch.arange(256) % 128 * (1 - torch.arange(256) // 128 * 2)).to(torch.int8)
    v = torch.arange(256).clamp(min=1).to(torch.uint8)
    m[255], v[255] = 127, 255
    state.m.copy_(m), state.v.copy_(v), state.bounds.fill_(1.0)
    grad[255] = 1.0  # with moments of 1 already: they stay
    for step in range(1, 2001):
        tokens.adamw([p], [grad], state, 1e-3, step, 0.9, beta2)
    want_m, want_v = m.int().clamp(-9, 9), v.int().clamp(max=last)
    want_m[255], want_v[255] = 127, 255
    assert torch.equal(state.m.cpu().int(), want_m) and torch.equal(state.v.cpu().int(), want_v)
    grad.zero_()
    for step in range(2001, 2101):
        tokens.adamw([p], [grad], state, 1e-3, step, 0.9, beta2)
    assert torch.equal(state.m.cpu().int(), want_m) and torch.equal(state.v.cpu().int(), want_v)
    want = torch.tensor([0.9**100, beta2**100], dtype=torch.float64)
    assert ((state.bounds[0].cpu().double() - want).abs() <= 101 * 2.0**-24 * want).all()  # a bound is rounded once a step
