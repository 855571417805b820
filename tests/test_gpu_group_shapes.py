"""Products grouped by rows at sizes that take every block of results and both ways of a sum (whole or in parts), with
blocks that a workgroup goes through one after another, tails of a sum, few and many groups, against 64 bits; layer norms of
more rows than workgroups."""
import pytest
import torch

from test_gpu_layers import TYPES, ln_check, mm_check, normal, offsets_of
from test_gpu_tokens import gen
from tile_differentiable_rasterizer_amd import tokens

pytestmark = pytest.mark.gpu

# rows, groups, k, n
SHAPES = [
    (1, 70, 8, 8), (1, 50, 664, 592), (29490, 57, 8, 8), (3, 6, 904, 1576), (26036, 18, 176, 8), (78, 87, 352, 1648), (2517, 13, 2776, 8), (8182, 18, 8, 8), (1, 56, 1792, 960),
    (35343, 79, 288, 8), (20038, 44, 8, 536), (12185, 23, 8, 1432), (3664, 6, 7232, 8), (17224, 1, 8, 8), (506, 22, 8, 2624), (1770, 81, 1104, 8), (31285, 71, 8, 144),
    (6378, 14, 8, 2424), (391, 17, 5952, 72), (9452, 2, 8, 2752), (17221, 2, 80, 400), (17303, 1, 4264, 8), (8631, 5, 8, 144), (17295, 4, 96, 8), (35689, 2, 136, 144),
    (876, 16, 168, 5080), (1386, 10, 6720, 144), (1689, 28, 6424, 144), (17270, 2, 8, 2016), (11817, 22, 144, 2944), (34408, 2, 8, 2112), (28111, 89, 72, 288),
    (10448, 1, 5448, 136), (7996, 16, 168, 4720), (9375, 35, 5568, 136), (7908, 26, 184, 5056), (5000, 70, 520, 264), (600, 66, 1032, 200), (30039, 1, 40, 96), (70001, 1, 136, 72),
]


def sizes_of(rows, groups, seed):
    """Uneven sizes that add up to rows less a few before and behind, every fifth one 0."""
    first, behind = (rows // 97, rows // 89) if rows > 200 else (0, 0)
    left = rows - first - behind
    share = torch.rand(groups, generator=torch.Generator().manual_seed(seed)).double() ** 2 + 0.05
    share[4::5] = 0
    at = [0, *((share.cumsum(0) / share.sum()) * left).round().int().tolist()]
    at[-1] = left
    return [b - a for a, b in zip(at, at[1:])], first, behind


def case(t, rows, groups, k, n, layout, off=0):
    """off: columns that wider matrices have before these."""
    g = gen(rows + groups)
    sizes, first, behind = sizes_of(rows, groups, rows)
    wide = lambda *s: normal(g, *s[:-1], s[-1] + 8 * (off > 0), t=TYPES[t])[..., off: off + s[-1]]  # noqa: E731
    x, dy = wide(rows, k), wide(rows, n)
    w = wide(groups, k, n) if layout == "kn" else wide(groups, n, k).transpose(1, 2)
    for m in (x, dy):
        m[:first] = torch.nan
        m[rows - behind:] = torch.inf
    return x, w, offsets_of(sizes, first), dy


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("rows, groups, k, n", SHAPES, ids=str)
def test_aligned(rows, groups, k, n, layout):
    mm_check(*case("bf16", rows, groups, k, n, layout))


# of these every block of the kernel that stages its tiles through registers
STAGED = [(1, 70, 8, 8), (1, 50, 664, 592), (29490, 57, 8, 8), (3, 6, 904, 1576), (26036, 18, 176, 8), (78, 87, 352, 1648), (2517, 13, 2776, 8), (1689, 28, 642, 145), (5000, 70, 7, 264),
          (4000, 3, 515, 5), (300, 2, 4105, 263), (9001, 1, 264, 129), (30039, 1, 40, 96),
          (70001, 1, 135, 72), (13, 1, 33, 40), (65, 4, 65, 9), (40, 2, 72, 31)]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows, groups, k, n", STAGED, ids=str)
def test_staged(rows, groups, k, n, t, off, layout):
    mm_check(*case(t, rows, groups, k, n, layout, off))


@pytest.mark.parametrize("t", TYPES)
def test_parts_in_graphs_on_one_workspace(t):
    """Sums in parts: two graphs that share a workspace, replayed one after another with eager calls between them."""
    sets = [case(t, 300, 2, 4104, 264, "kn"), case(t, 260, 3, 4104, 264, "nk")]
    need = lambda s: tokens.GsGroupMM(s[0].shape[0], 4104, 264, s[1].shape[0], tokens.TYPES[s[0].dtype], s[2].data_ptr())  # noqa: E731
    size = max(max(tokens.lib().gs_group_mm_fwd_workspace_bytes(need(s)), tokens.lib().gs_group_mm_bwd_workspace_bytes(need(s))) for s in sets)
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    run = lambda x, w, offs, dy: [tokens.group_mm_fwd(x, w, offs, workspace=ws), *tokens.group_mm_bwd(dy, x, w, offs, workspace=ws)]  # noqa: E731
    want = [[z.clone() for z in run(*s)] for s in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run(*s))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        for z in got[i]:
            z.fill_(7.0)
        graphs[i].replay()
        eager = run(*sets[1 - i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])) and all(torch.equal(a, b) for a, b in zip(eager, want[1 - i])), i


def test_parts_on_two_streams():
    """Calls beside each other, each with parts of its own."""
    sets = [case("bf16", 300, 2, 4104, 264, "kn"), case("f32", 260, 3, 4104, 264, "nk")]
    run = lambda x, w, offs, dy: [tokens.group_mm_fwd(x, w, offs), *tokens.group_mm_bwd(dy, x, w, offs)]  # noqa: E731
    want = [run(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for once in got[i] for a, b in zip(once, want[i])), i


def test_offsets_that_decrease():
    """More rows by their spans than there are: what is written lies inside, the call ends, and the next one is right."""
    x, w, offs, dy = case("bf16", 5000, 8, 256, 512, "kn")
    want = tokens.group_mm_fwd(x, w, offs)
    room = torch.full((5002, 512), 3.0, dtype=x.dtype, device="cuda")
    for bad in ([5000, 0] * 4 + [5000], [0, 5000, -5, 5000, 0, 2**31 - 1, 0, 5000, 0], [4000, 3999] * 4 + [0]):
        tokens.group_mm_fwd(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=room[1:-1])
        tokens.group_mm_bwd(dy, x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    assert (room[0] == 3).all() and (room[-1] == 3).all() and torch.equal(tokens.group_mm_fwd(x, w, offs), want)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows, width", [(40000, 24), (20000, 200), (9000, 400), (17000, 600), (3000, 600), (2500, 1500), (2100, 2500), (2100, 5000), (2100, 9000)])
def test_layer_norm_of_many_rows(rows, width, t):
    g = gen(rows)
    ln_check(normal(g, rows, width, t=TYPES[t]), normal(g, width) + 1, normal(g, width), 1e-5, normal(g, rows, width, t=TYPES[t]))
