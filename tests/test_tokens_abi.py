"""CPU-side checks of the token operators' C ABI (include/gs_tokens.h): the library exports what
the header declares, refuses bad arguments before any HIP call, and sizes workspaces."""
import ctypes as C
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gs_tokens.h")
LIB = os.path.join(ROOT, "tile_differentiable_rasterizer_amd", "libgsraster.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libgsraster.so not built")

OK, BAD, OVERFLOW, WORKSPACE = 0, 1, 3, 5
A = 1 << 20  # an aligned stand-in, never dereferenced


def tokens():
    from tile_differentiable_rasterizer_amd import tokens as t

    return t


def test_header_and_binding_name_the_same_calls():
    t = tokens()
    names = set(re.findall(r"^\s*(?:gs_status|size_t)\s+(gs_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(t.EXPORTS)
    lib = C.CDLL(LIB)
    for n in names:
        assert hasattr(lib, n), n


def heads(data=A, b=4096, tok=512, h=64):
    return tokens().GsHeads(data, b, tok, h)


def norm_call(data=A, heads_of=None, w=A, table=A, bwd=False, ws=A, ws_bytes=1 << 30, dw=A, **change):
    t = tokens()
    s = dict(batch=2, q_len=3, k_len=5, q_heads=4, k_heads=2, head_dim=64, rot_dim=32, pairs=0, type=0, eps=1e-6, n_pos=9)
    s.update(change)
    p = t.GsNormRotate(**s)
    x = heads_of or heads(data)
    L = t.lib()
    if bwd:
        return L.gs_norm_rotate_bwd(p, x, x, x, x, w, w, table, table, None, None, x, x, dw, dw, ws, ws_bytes, None)
    return L.gs_norm_rotate_fwd(p, x, x, w, w, table, table, None, None, x, x, None)


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=A + 8), dict(heads_of=(A, 4, 512, 64)), dict(heads_of=(A, 4096, -8, 64)),
                                 dict(w=None), dict(w=A + 4), dict(table=None), dict(table=A + 8), dict(n_pos=0), dict(head_dim=4), dict(head_dim=60),
                                 dict(head_dim=264), dict(rot_dim=72), dict(rot_dim=12), dict(rot_dim=-8), dict(pairs=2), dict(type=2),
                                 dict(type=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(batch=-1), dict(q_len=-1), dict(k_heads=-1)])
@pytest.mark.parametrize("bwd", [False, True])
def test_norm_rotate_refuses(bad, bwd):
    if "heads_of" in bad:
        bad = dict(heads_of=tokens().GsHeads(*bad["heads_of"]))
    assert norm_call(bwd=bwd, **bad) == BAD


def test_norm_rotate_limits():
    assert norm_call(q_len=1 << 31) == OVERFLOW
    assert norm_call(k_len=1 << 62) == OVERFLOW
    assert norm_call(bwd=True, dw=None) == BAD
    assert norm_call(bwd=True, ws=None) == WORKSPACE
    assert norm_call(bwd=True, ws=A + 8) == WORKSPACE
    assert norm_call(bwd=True, ws_bytes=100) == WORKSPACE
    assert norm_call(batch=0, data=None) == OK  # nothing to do: no pointer is looked at, nothing launched
    assert norm_call(q_len=0, k_len=0, data=None, w=None, table=None) == OK
    t = tokens()
    p = t.GsNormRotate(1, 1, 1, 8, 8, 64, 64, 0, 0, 1e-6, 8)
    assert 0 < t.lib().gs_norm_rotate_workspace_bytes(p) < 1 << 20
    p.head_dim = 7
    assert t.lib().gs_norm_rotate_workspace_bytes(p) == 0
    assert t.lib().gs_norm_rotate_workspace_bytes(None) == 0


def attn_call(data=A, kv=None, bwd=False, lse=A, ws=A, ws_bytes=1 << 40, **change):
    t = tokens()
    s = dict(batch=2, q_len=7, k_len=9, q_heads=4, kv_heads=2, head_dim=64, type=0, scale=0.125)
    s.update(change)
    p = t.GsCrossAttn(**s)
    x = heads(data)
    y = kv or x
    L = t.lib()
    if bwd:
        return L.gs_cross_attn_bwd(p, x, x, y, y, x, lse, x, y, y, ws, ws_bytes, None)
    return L.gs_cross_attn_fwd(p, x, y, y, x, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=A + 4), dict(kv=(A, 1, 512, 64)), dict(kv=(A, 4096, 516, 64)), dict(kv=(A, 4096, 512, -64)),
                                 dict(q_heads=3), dict(q_heads=0), dict(kv_heads=0), dict(kv_heads=-2), dict(head_dim=0), dict(head_dim=36),
                                 dict(head_dim=136), dict(type=3), dict(scale=float("inf")), dict(scale=float("nan")), dict(batch=-1),
                                 dict(q_len=-1), dict(k_len=-1), dict(ranges=A + 2), dict(ranges=A, ranges_row_stride=-1),
                                 dict(ranges=A, ranges_batch_stride=-1), dict(key_mask=A, key_mask_batch_stride=-1), dict(lse=A + 2)])
@pytest.mark.parametrize("bwd", [False, True])
def test_cross_attn_refuses(bad, bwd):
    if "kv" in bad:
        bad = dict(kv=tokens().GsHeads(*bad["kv"]))
    assert attn_call(bwd=bwd, **bad) == BAD


def test_cross_attn_limits():
    assert attn_call(q_len=1 << 31) == OVERFLOW
    assert attn_call(k_len=1 << 31) == OVERFLOW
    assert attn_call(batch=1 << 31) == OVERFLOW
    assert attn_call(batch=1 << 61, k_len=1 << 62) == OVERFLOW
    assert attn_call(k_len=100_000, ws=None) == WORKSPACE  # a long axis for few rows: parts
    assert attn_call(k_len=100_000, ws=A + 8) == WORKSPACE
    assert attn_call(k_len=100_000, ws_bytes=64) == WORKSPACE
    assert attn_call(bwd=True, lse=None) == BAD
    assert attn_call(bwd=True, ws=None) == WORKSPACE
    assert attn_call(bwd=True, ws_bytes=16) == WORKSPACE
    assert attn_call(batch=0, data=None) == OK
    assert attn_call(q_len=0, data=None, kv=heads()) == OK
    assert attn_call(batch=0, data=None, lse=None, ws=None, bwd=True) == OK
    L = tokens().lib()
    p = tokens().GsCrossAttn(batch=8, q_len=1, k_len=65280, q_heads=32, kv_heads=4, head_dim=128, type=0, scale=1.0)
    few = L.gs_cross_attn_fwd_workspace_bytes(p)
    assert 0 < few < 1 << 27
    p.q_len = 1 << 16
    assert L.gs_cross_attn_fwd_workspace_bytes(p) == 0  # rows enough: nothing is split
    assert L.gs_cross_attn_bwd_workspace_bytes(p) >= 8 * 32 * 4 << 16
    p.head_dim = 12
    assert L.gs_cross_attn_bwd_workspace_bytes(p) == 0
    assert L.gs_cross_attn_fwd_workspace_bytes(None) == 0


def test_cross_attn_orders_nothing_without_keys():
    """Rows are put in order by the key tiles they see: of none, as many rows as there may be."""
    p = tokens().GsCrossAttn(batch=1, q_len=1 << 23, k_len=1, q_heads=32, kv_heads=32, head_dim=8, type=0, scale=1.0, ranges=A, ranges_row_stride=1)
    L = tokens().lib()
    assert L.gs_cross_attn_fwd_workspace_bytes(p) == 8 << 16
    p.k_len = 0
    assert L.gs_cross_attn_fwd_workspace_bytes(p) == 0


def gate_call(rows=3, width=64, act=0, type=0, x=A, stride=64, codes=A, bounds=A, bwd=False):
    L = tokens().lib()
    if bwd:
        return L.gs_gate8_bwd(rows, width, act, type, x, stride, codes, bounds, x, stride, x, stride, None, 0, None)
    return L.gs_gate8_fwd(rows, width, act, type, x, stride, x, stride, x, stride, codes, bounds, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=A + 1), dict(type=1, x=A + 2), dict(stride=63), dict(stride=-64), dict(codes=None),
                                 dict(bounds=None), dict(bounds=A + 4), dict(act=2), dict(act=-1), dict(type=2), dict(rows=-1), dict(width=-1)])
@pytest.mark.parametrize("bwd", [False, True])
def test_gate8_refuses(bad, bwd):
    assert gate_call(bwd=bwd, **bad) == BAD


def test_gate8_limits():
    for bwd in (False, True):
        assert gate_call(rows=1 << 31, bwd=bwd) == OVERFLOW
        assert gate_call(rows=1 << 30, width=1 << 10, stride=1 << 10, bwd=bwd) == OVERFLOW
        assert gate_call(width=1 << 62, stride=1 << 62, bwd=bwd) == OVERFLOW
        assert gate_call(rows=0, x=None, codes=None, bounds=None, bwd=bwd) == OK
        assert gate_call(width=0, stride=0, x=None, codes=None, bounds=None, bwd=bwd) == OK


def test_binding_refuses_what_the_c_calls_cannot_see():
    import torch

    t = tokens()
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError):  # not on the GPU
        t.cross_attn_fwd(q, q, q)
    with pytest.raises(ValueError):  # another head size
        t.cross_attn_fwd(q, torch.zeros(1, 2, 4, 32), torch.zeros(1, 2, 4, 32))
    with pytest.raises(ValueError):
        t.norm_rotate_fwd(q, q, torch.ones(64), torch.ones(64), torch.ones(2, 32), torch.ones(2, 32))
    with pytest.raises(ValueError):
        t.gate8_fwd(torch.zeros(2, 8), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        t.gate8_fwd(torch.zeros(2, 8), torch.zeros(2, 8), act="relu")
    with pytest.raises(ValueError):
        t.gate8_fwd(torch.zeros(2, 8, dtype=torch.float16), torch.zeros(2, 8, dtype=torch.float16))


@pytest.mark.parametrize("bwd", [False, True])
def test_cross_attn_refuses_a_scale_past_its_exponent(bwd):
    """The kernels work in base 2: scale * log2(e) has to be a float32."""
    for scale in (3e38, -2.4e38):
        assert attn_call(bwd=bwd, scale=scale) == BAD
    for scale in (2.3e38, -2.3e38, 0.0, 1e-45):
        assert attn_call(bwd=bwd, scale=scale, batch=0) == OK


OVERLAPS = [dict(b=0), dict(tok=0), dict(h=0), dict(b=32), dict(tok=56), dict(h=8)]


@pytest.mark.parametrize("over", OVERLAPS, ids=str)
def test_outputs_whose_vectors_overlap_are_refused(over):
    """An input may repeat its vectors (a stride of 0); an output that did would hold whichever came last.  Nothing is
    launched: the calls that are not refused have a workspace that is too small, or nothing to do."""
    t = tokens()
    L, x, bad = t.lib(), heads(), heads(**over)
    n = t.GsNormRotate(batch=2, q_len=3, k_len=5, q_heads=4, k_heads=2, head_dim=64, rot_dim=32, pairs=0, type=0, eps=1e-6, n_pos=9)
    a = t.GsCrossAttn(batch=2, q_len=7, k_len=9, q_heads=4, kv_heads=2, head_dim=64, type=0, scale=0.125)
    for i in range(2):
        o = [bad if j == i else x for j in range(2)]
        assert L.gs_norm_rotate_fwd(n, x, x, A, A, A, A, None, None, *o, None) == BAD
        assert L.gs_norm_rotate_bwd(n, x, x, x, x, A, A, A, A, None, None, *o, A, A, A, 1 << 30, None) == BAD
    assert L.gs_cross_attn_fwd(a, x, x, x, bad, A, A, 1 << 40, None) == BAD
    for i in range(3):
        o = [bad if j == i else x for j in range(3)]
        assert L.gs_cross_attn_bwd(a, x, x, x, x, x, A, *o, A, 1 << 40, None) == BAD
    assert L.gs_cross_attn_bwd(a, bad, bad, bad, bad, bad, A, x, x, x, A, 16, None) == WORKSPACE  # as inputs
    assert L.gs_norm_rotate_bwd(n, bad, bad, bad, bad, A, A, A, A, None, None, x, x, A, A, A, 16, None) == WORKSPACE
    # axes of length 1 have no stride
    n.batch = n.q_len = n.k_len = n.q_heads = n.k_heads = 1
    assert L.gs_norm_rotate_bwd(n, x, x, x, x, A, A, A, A, None, None, bad, bad, A, A, A, 16, None) == WORKSPACE
    a.batch = a.q_len = a.k_len = a.q_heads = a.kv_heads = 1
    assert L.gs_cross_attn_bwd(a, x, x, x, x, x, A, bad, bad, bad, A, 16, None) == WORKSPACE
