"""Products grouped by rows with weights that repeat along an axis (a stride of 0), against 64 bits (tolerances: test_gpu_layers)."""
import pytest
import torch

from test_gpu_layers import TYPES, close, mm_case, mm_check
from test_gpu_tokens import gen, half_step, normal
from tile_differentiable_rasterizer_amd import tokens

pytestmark = pytest.mark.gpu

SHAPES = [([30, 0, 50], 64, 40), ([130, 7, 64], 136, 264), ([3, 1, 2], 5, 7), ([40, 9, 1], 65, 1), ([40, 9, 1], 1, 65), ([300, 200, 100], 363, 250)]
REPEATS = {"rows": lambda w: w[:, :1].expand_as(w), "columns": lambda w: w[:, :, :1].expand_as(w), "groups and rows": lambda w: w[:1, :1].expand_as(w),
           "rows of a transposed one": lambda w: w.transpose(1, 2).contiguous().transpose(1, 2)[:, :, :1].expand_as(w)}


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("which", REPEATS)
@pytest.mark.parametrize("sizes, k, n", SHAPES, ids=str)
def test_weights_that_repeat(sizes, k, n, which, t):
    x, w, offs, dy = mm_case(t, sizes, k, n, first=1, behind=2)
    w = REPEATS[which](w)
    if w.stride(1) != 1 and w.stride(2) != 1 and k > 1 and n > 1:  # (the column of a matrix whose rows are dense)
        with pytest.raises(ValueError, match="dense"):
            tokens.group_mm_fwd(x, w, offs)
        return
    mm_check(x, w, offs, dy, which)


@pytest.mark.parametrize("t", TYPES)
def test_gradient_of_a_row_that_all_share(t):
    """The gradient of what repeats is the sum over its copies."""
    x, w, offs, dy = mm_case(t, [30, 0, 50], 64, 40)
    row = normal(gen(5), 40, t=TYPES[t]).requires_grad_()
    tokens.group_mm(x, row.expand(3, 64, 40), offs).backward(dy)
    parts = tokens.group_mm_bwd(dy, x, row.detach().expand(3, 64, 40), offs)[1].double()
    terms = parts.shape[0] * parts.shape[1]
    close(row.grad, parts.sum((0, 1)), terms * half_step(x.dtype) * parts.abs().sum((0, 1)), "shared")
