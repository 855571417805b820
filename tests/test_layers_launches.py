"""CPU-side checks of what the operators that train a decoder layer launch, with the stand-in for HIP's launch calls:
nothing after a launch that failed, grids that HIP takes up to the documented limits, workspaces that are too small."""
import json
import os
import subprocess
import sys

import pytest

from test_layers_abi import group_call, layer_norm_call
from test_tokens_abi import A, LIB, tokens
from test_tokens_launches import CHILD, HIP, OK, OVERFLOW, STAND_IN

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgsraster.so not built")

WORKSPACE = 5


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    """calls [(function of test_layers_abi, its arguments, the launch that fails or -1)] -> [(status, workgroups of each launch)]"""
    where = tmp_path_factory.mktemp("stand_in")
    (where / "hip.c").write_text(STAND_IN)
    subprocess.run(["gcc", "-O1", "-fPIC", "-shared", "-o", str(where / "hip.so"), str(where / "hip.c")], check=True)
    tests = os.path.dirname(os.path.abspath(__file__))
    child = subprocess.Popen([sys.executable, "-c", CHILD.replace("import test_tokens_abi as abi", "import test_layers_abi as abi"), str(where / "hip.so"), tests,
                              os.path.dirname(tests)], stdin=subprocess.PIPE, stdout=subprocess.PIPE, text=True)

    def run(calls):
        child.stdin.write(json.dumps(calls) + "\n")
        child.stdin.flush()
        line = child.stdout.readline()
        assert line, "the process ended"
        return json.loads(line)

    yield run
    child.stdin.close()
    assert child.wait(60) == 0


# long sums with few results, in parts: dx's and dW's
PARTS = dict(rows=20, k=264, n=4104, groups=1)
PARTS_DW = dict(rows=8000, k=512, n=512, groups=1)
CHAINS = [("layer_norm_call", dict(rows=5000, bwd=True), 2), ("group_call", dict(PARTS, k=4104, n=264), 2), ("group_call", dict(PARTS, bwd=True), 3),
          ("group_call", dict(PARTS_DW, bwd=True), 3), ("group_call", dict(PARTS_DW, type=1, bwd=True), 3), ("group_call", dict(PARTS_DW, k=511, bwd=True), 3),
          ("group_call", dict(rows=64, k=512, n=512, groups=4, bwd=True), 2), ("adamw_call", dict(n=[300] * 200), 4), ("adamw_call", dict(n=[0] * 100 + [1] * 65, bits=32), 2)]


@pytest.mark.parametrize("call, how, count", CHAINS, ids=str)
def test_nothing_follows_a_failed_launch(launched, call, how, count):
    got = launched([(call, how, i) for i in range(-1, 6)])
    status, every = got[0]
    assert status == OK and len(every) == count and min(every) > 0
    for i, (status, launches) in enumerate(got[1: count + 1]):
        assert status == HIP and len(launches) == i + 1, f"launch {i} fails, {len(launches)} are made"


@pytest.mark.parametrize("type", [0, 1])
@pytest.mark.parametrize("bwd", [False, True])
def test_grids_of_the_products(launched, bwd, type):
    """Each side of the limit of 2^23 blocks of 128 x 64, aligned and not; the most groups and rows."""
    most = 1 << 23
    # by rows a block more for each span
    inside = [dict(rows=(most - 4) * 128, k=64, n=64, groups=1), dict(rows=(most - 4) * 128, k=63, n=61, groups=1), dict(rows=1 << 20, k=64, n=64, groups=65536),
              dict(rows=100, k=(1 << 24), n=8, groups=2), dict(rows=100, k=8, n=1 << 24, groups=2), dict(rows=64, k=13, n=1 << 24, groups=3), dict(rows=100, k=72, n=1 << 24, groups=28)]
    outside = [dict(rows=(most - 2) * 128, k=64, n=64, groups=1), dict(rows=1 << 20, k=64 * 128, n=64 * 128, groups=65536), dict(rows=(1 << 31) - 256, k=8, n=8, groups=1),
               dict(rows=100, k=72, n=1 << 24, groups=32)]
    for how, (status, launches) in zip(inside, launched([("group_call", dict(how, type=type, bwd=bwd), -1) for how in inside])):
        assert status == OK and launches and min(launches) > 0, how
    for how, (status, launches) in zip(outside, launched([("group_call", dict(how, type=type, bwd=bwd), -1) for how in outside])):
        assert status == OVERFLOW and not launches, how


def test_grids_of_the_layer_norm(launched):
    hows = [dict(rows=(1 << 31) - 1, width=w, stride=w, y_stride=w, dy_stride=w, bwd=b, type=t) for w in (1, 64, 130, 400, 1000, 2000, 4000, 8000, 16384) for b in (False, True) for t in (0, 1)]
    for how, (status, launches) in zip(hows, launched([("layer_norm_call", how, -1) for how in hows])):
        assert status == OK and len(launches) == 1 + how["bwd"] and min(launches) > 0, how
    [(status, launches)] = launched([("layer_norm_call", dict(rows=0, width=16384, bwd=True), -1)])
    assert status == OK and launches == [64]


@pytest.mark.parametrize("bits", [8, 32])
def test_grids_of_adamw(launched, bits):
    """2^34 units and more are refused, whichever way they are spread; a call of many tensors goes in launches of 64."""
    most = 1 << 34
    inside = [[most - 256], [most // 2, most // 2 - 256], [1] * 64 + [most // 2], [(1 << 24) - 257] * 3]
    outside = [[most], [most - 256, 1], [most // 2 + 1, most // 2 - 256, 0]]
    for n, (status, launches) in zip(inside, launched([("adamw_call", dict(n=n, bits=bits), -1) for n in inside])):
        assert status == OK and len(launches) == -(-len(n) // 64) and min(launches) > 0
    for n, (status, launches) in zip(outside, launched([("adamw_call", dict(n=n, bits=bits), -1) for n in outside])):
        assert status == OVERFLOW and not launches


def test_grids_of_the_moments(launched):
    got = launched([("moments_call", dict(blocks=n), -1) for n in (1, (1 << 26) - 1, 1 << 26, (1 << 27) - 1)])
    assert [status for status, _ in got] == [OK, OK, OVERFLOW, OVERFLOW] and all(min(launches) > 0 for _, launches in got[:2])


@pytest.mark.parametrize("how", [dict(rows=20, k=4104, n=264, groups=1), dict(rows=20, k=264, n=4104, groups=1, bwd=True), dict(rows=8000, k=512, n=512, groups=1, bwd=True),
                                 dict(rows=8000, k=511, n=513, groups=1, bwd=True), dict(rows=800, k=512, n=1024, groups=4, type=1, bwd=True)], ids=str)
def test_products_want_their_workspace(how):
    t = tokens()
    size = t.lib().gs_group_mm_bwd_workspace_bytes if how.get("bwd") else t.lib().gs_group_mm_fwd_workspace_bytes
    need = size(t.GsGroupMM(**{"type": 0, "offsets": A, **{k: v for k, v in how.items() if k != "bwd"}}))
    assert need > 0 and need % 16 == 0
    for bad in (dict(ws=None), dict(ws=A + 8), dict(ws_bytes=need - 1)):
        assert group_call(**how, **bad) == WORKSPACE


def test_products_workspace_is_bounded():
    """Parts are made where results are few: at most 256 of them, and of a launch's blocks."""
    t = tokens()
    for rows in (1, 100, 5000, 1 << 20, 1 << 26):
        for k, n in ((8, 8), (512, 512), (8192, 264), (264, 8192), (1 << 20, 8)):
            for groups in (1, 16, 500):
                p = t.GsGroupMM(rows, k, n, groups, 0, A)
                assert t.lib().gs_group_mm_fwd_workspace_bytes(p) <= 1 << 28 and t.lib().gs_group_mm_bwd_workspace_bytes(p) <= 1 << 28, (rows, k, n, groups)


def test_layer_norm_of_one_workgroup_wants_none():
    assert layer_norm_call(bwd=True, rows=0, ws=None) != WORKSPACE and tokens().lib().gs_layer_norm_workspace_bytes(16, 64) == 0


@pytest.mark.parametrize("type", [0, 1])
def test_weights_that_repeat(launched, type):
    """Weights, as an input, may repeat along any axis but the dense one; as an output they may not."""
    hows = [dict(w_strides=s, k=k, n=n) for s, k, n in (((0, 96, 1), 64, 96), ((6144, 0, 1), 64, 96), ((0, 0, 1), 64, 96), ((6144, 1, 0), 64, 96), ((64, 1, 0), 64, 96), ((96, 0, 1), 64, 96),
                                                        ((64, 1, 0), 64, 1), ((1, 0, 0), 1, 96), ((1, 0, 0), 64, 1), ((0, 0, 0), 1, 1))]
    for how, (status, launches) in zip(hows, launched([("group_call", dict(how, type=type), -1) for how in hows])):
        assert status == OK and launches, how
    for how, (status, launches) in zip(hows, launched([("group_call", dict(how, type=type, bwd=True, dw=None), -1) for how in hows])):
        assert status == OK and launches, how
    hows = [how for how in hows if (how["w_strides"], how["n"]) != ((64, 1, 0), 1)]  # (an axis of length 1)
    for how, (status, _) in zip(hows, launched([("group_call", dict(how, type=type, bwd=True, w_strides=None, dw_strides=how["w_strides"]), -1) for how in hows])):
        assert status == 1, how
