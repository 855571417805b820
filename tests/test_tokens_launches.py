"""CPU-side checks of what the token operators launch: a small library that stands in for HIP's launch
calls counts them, refuses a grid that HIP refuses, and fails a launch where a test asks for it.

The stand-in is loaded before libgsraster in a process of its own, so that the library's launches
reach it; no kernel runs."""
import json
import os
import subprocess
import sys

import pytest

from test_tokens_abi import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgsraster.so not built")

OK, OVERFLOW, HIP = 0, 3, 4

# hipLaunchKernel takes grids of fewer than 2^32 work items an axis
STAND_IN = """
#include <stddef.h>
#include <stdint.h>
typedef struct { uint32_t x, y, z; } dim3;
int fail_at = -1, launches = 0, last = 0;
double workgroups[64];
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t lds, void* stream) {
  int fits = (uint64_t)g.x * b.x >> 32 == 0 && (uint64_t)g.y * b.y >> 32 == 0 && g.x && g.y && g.z;
  if (launches < 64) workgroups[launches] = fits ? (double)g.x * g.y * g.z : -1.0;
  if (!fits || launches == fail_at) last = 9;
  return launches++ == fail_at || !fits ? 9 : 0;
}
static dim3 grid, block;
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void* stream) { grid = g; block = b; return 0; }
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* lds, void** stream) {
  *g = grid; *b = block; *lds = 0; *stream = 0;
  return 0;
}
int hipGetLastError(void) { int e = last; last = 0; return e; }
"""

CHILD = """
import ctypes, json, sys
stand_in = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path[:0] = sys.argv[2:4]
import test_tokens_abi as abi
var = lambda name, t=ctypes.c_int: t.in_dll(stand_in, name)
for line in sys.stdin:
    out = []
    for call, how, fail_at in json.loads(line):
        var("fail_at").value, var("launches").value, var("last").value = fail_at, 0, 0
        status = getattr(abi, call)(**how)
        n = var("launches").value
        out.append((status, list(var("workgroups", ctypes.c_double * 64)[:n])))
    print(json.dumps(out), flush=True)
"""


@pytest.fixture(scope="module")
def launched(tmp_path_factory):
    """calls [(function of test_tokens_abi, its arguments, the launch that fails or -1)] -> [(status, workgroups of each launch)]"""
    where = tmp_path_factory.mktemp("stand_in")
    (where / "hip.c").write_text(STAND_IN)
    subprocess.run(["gcc", "-O1", "-fPIC", "-shared", "-o", str(where / "hip.so"), str(where / "hip.c")], check=True)

    tests = os.path.dirname(os.path.abspath(__file__))
    child = subprocess.Popen([sys.executable, "-c", CHILD, str(where / "hip.so"), tests, os.path.dirname(tests)], stdin=subprocess.PIPE,
                             stdout=subprocess.PIPE, text=True)

    def run(calls):
        child.stdin.write(json.dumps(calls) + "\n")
        child.stdin.flush()
        line = child.stdout.readline()
        assert line, "the process ended"
        return json.loads(line)

    yield run
    child.stdin.close()
    assert child.wait(60) == 0


A = 1 << 20
# rows with ranges of their own from 2^28 pairs on (ordered), and long axes that are split and joined
ORDERED = dict(batch=2, q_len=4200, k_len=2100, q_heads=16, kv_heads=16, head_dim=32, ranges=A, ranges_batch_stride=4200, ranges_row_stride=1)
SPLIT_KEYS, SPLIT_ROWS = dict(batch=1, q_len=4, k_len=9000), dict(batch=1, q_len=9000, k_len=4)
CHAINS = [("attn_call", SPLIT_KEYS), ("attn_call", ORDERED), ("attn_call", dict(SPLIT_KEYS, bwd=True)), ("attn_call", dict(SPLIT_ROWS, bwd=True)),
          ("attn_call", dict(ORDERED, bwd=True)), ("norm_call", dict(bwd=True))]


@pytest.mark.parametrize("call, how", CHAINS, ids=str)
def test_nothing_follows_a_failed_launch(launched, call, how):
    """Kernels read what the ones before them leave (the rows' tiles, lengths, parts): after a launch that failed none is made."""
    got = launched([(call, how, i) for i in range(-1, 5)])
    status, every = got[0]
    assert status == OK and len(every) >= 2
    for i, (status, launches) in enumerate(got[1: len(every) + 1]):
        assert status == HIP and len(launches) == i + 1, f"launch {i} fails, {len(launches)} are made"


@pytest.mark.parametrize("bwd", [False, True])
def test_grids_of_the_gate(launched, bwd):
    """Blocks up to 2^31 are taken, on grids that HIP takes, eight a workgroup; the strides are the width's."""
    blocks = [(1 << 27) - 1, 1 << 27, (1 << 27) + 1, (1 << 30) + 12345, (1 << 31) - 1]
    got = launched([("gate_call", dict(rows=n, width=8, stride=8, bwd=bwd), -1) for n in blocks])
    for n, (status, launches) in zip(blocks, got):
        assert status == OK and len(launches) == 1 and -(-n // 8) <= launches[0] < -(-n // 8) + 256, n
    wide = launched([("gate_call", dict(rows=2, width=(1 << 30) * 256, stride=(1 << 30) * 256, bwd=bwd), -1),
                     ("gate_call", dict(rows=1, width=(1 << 30) * 256 + 1, stride=0, bwd=bwd), -1)])
    assert wide[0][0] == OVERFLOW and wide[1][0] == OK


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("how", [dict(batch=(1 << 24) - 1), dict(batch=1 << 20, q_heads=16, kv_heads=16), dict(batch=1 << 20, q_heads=8, kv_heads=8, q_len=129),
                                 dict(batch=1 << 20, q_heads=32, kv_heads=8, k_len=129), dict(batch=1 << 30), dict(batch=1, q_len=(1 << 31) - 129, k_len=1)], ids=str)
def test_grids_of_the_attention(launched, how, bwd):
    """2^24 blocks of 128 rows (back: or keys) are one more than a grid of 256 threads each takes: refused before any launch."""
    how = {**dict(q_len=1, k_len=1, q_heads=1, kv_heads=1, head_dim=8), **how}
    rows = how["q_len"] * how["q_heads"] // how["kv_heads"]
    blocks = how["batch"] * how["kv_heads"] * -(-max(rows, how["k_len"] if bwd else 0) // 128)
    [(status, launches)] = launched([("attn_call", dict(how, bwd=bwd), -1)])
    if blocks < 1 << 24:
        assert status == OK and launches and min(launches) > 0
    else:
        assert status == OVERFLOW and not launches


def test_grids_of_the_norm(launched):
    how = dict(batch=1, q_len=(1 << 31) - 1, k_len=(1 << 31) - 1, q_heads=1, k_heads=1, head_dim=256, n_pos=5)
    for status, launches in launched([("norm_call", how, -1), ("norm_call", dict(how, bwd=True), -1)]):
        assert status == OK and min(launches) > 0
