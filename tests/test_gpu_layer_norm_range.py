"""Layer norm of rows far from 0, up to the ends of what the header states, against 64 bits (tolerances: test_gpu_layers)."""
import pytest
import torch

from test_gpu_layers import ln_check
from test_gpu_tokens import TYPES, U, close, gen, half_step, normal
from tile_differentiable_rasterizer_amd import tokens

pytestmark = pytest.mark.gpu

WIDTHS = [5, 300, 700, 1500, 2500, 4096, 5000, 9001, 16384]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_rows_whose_sum_is_no_float32(t, width):
    """Rows of one value up to 3e38, whose sums pass float32's largest number."""
    g, t = gen(width), TYPES[t]
    values = [1e30, 3e34, -1e36, 1e37, 3e38, -3e38]
    x = torch.tensor(values, device="cuda").to(t)[:, None].expand(len(values), width).contiguous()
    w, b, dy = normal(g, width), normal(g, width), normal(g, len(values), width, t=t)
    y, (dx, dw, db) = tokens.layer_norm_fwd(x, w, b), tokens.layer_norm_bwd(dy, x, w)
    # The definition, with a distance of 0 from the mean: a mean in float64 is off by 2^-53 of 3e38, whose square is 1e45 and not 0, so
    # it is no reference here.  A mean that float32 does not hold is off by 7e22 and more (half a spacing of 1e30 is 4e22), whose square
    # is infinite: 1 / sqrt of it is 0, xh is 0 as it is without, and dx is 0 where the formula has (g - mean(g)) / sqrt(eps).
    assert torch.equal(y, b.to(t).expand_as(y)) and (dw == 0).all()
    gw = dy.double() * w.double()
    mean, size = gw.mean(-1, keepdim=True), gw.abs().mean(-1, keepdim=True)
    full = (gw - mean) / 1e-5**0.5
    for row in range(len(values)):
        if (dx[row] != 0).any():
            tol = (40 * U * size[row] + 4 * U * (gw[row].abs() + mean[row].abs())) / 1e-5**0.5 + (8 * U + half_step(t)) * full[row].abs()
            close(dx[row], full[row], tol, f"dx of {values[row]}")
    close(db, dy.double().sum(0), 96 * U * dy.double().abs().sum(0), "db")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_mixed_with_ordinary_rows(t, width):
    """Rows of ordinary size beside them keep their bits."""
    g, t = gen(width + 1), TYPES[t]
    x, dy, w = normal(g, 12, width, t=t), normal(g, 12, width, t=t), normal(g, width)
    y, dx = tokens.layer_norm_fwd(x, w), tokens.layer_norm_bwd(dy, x, w)[0]
    far = x.clone()
    far[::3] = 2e38
    keep = [i for i in range(12) if i % 3]
    assert torch.equal(tokens.layer_norm_fwd(far, w)[keep], y[keep]) and torch.equal(tokens.layer_norm_bwd(dy, far, w)[0][keep], dx[keep])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows, width", [(12287, 800), (12288, 800), (12289, 1024), (12290, 1300), (12300, 2047), (12301, 2048), (12302, 600)])
def test_many_rows_by_workgroups(rows, width, t):
    """Each side of where the backward pass takes more workgroups."""
    g = gen(rows)
    ln_check(normal(g, rows, width, t=TYPES[t]), normal(g, width) + 1, None, 1e-5, normal(g, rows, width, t=TYPES[t]))
