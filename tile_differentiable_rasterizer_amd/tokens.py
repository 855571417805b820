"""ctypes binding of libgsraster's token operators (the C ABI in include/gs_tokens.h).

The parts of a decoder layer that predicts Gaussians from images which are not plain matrix
products: norms of queries and keys with the position rotation, attention of the tokens to the
encoder's states, and the gated activation that keeps its inputs as 8-bit codes.  And what trains
such layers beside them: layer norm, the products of rows with their group's weights (experts), and
AdamW over all tensors at once.

Tensors are bfloat16 or float32 on the GPU, laid out as include/gs_tokens.h says: vectors dense in
their last axis, on 16-byte boundaries, any strides else (views of one projection's output are
taken as they are; layer_norm and group_mm take any alignment).  Shapes and types are checked here (the C calls do not see them: ValueError),
everything else by the C calls (raster.GsError).  Work goes to the current stream of the tensors' GPU, or to
``stream``, which is one of that GPU; outputs and workspaces that are not given are torch tensors made on that same stream
(a workspace is given back to torch when the call returns, in stream order).

``norm_rotate``, ``cross_attention``, ``gated8``, ``layer_norm`` and ``group_mm`` are the same operators as
differentiable torch functions.  Their gradients come from C calls that torch does not record: second
derivatives through them are an error (``once``).  Calls and functions may be captured into a graph (lr and step of ``adamw`` as they were then);
torch's own rule for a captured ``backward()`` holds: no graph made before, on another stream, may still hold the same leaves.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import operator
import struct
from array import array

import torch

from . import raster
from .raster import _check

BF16, F32 = 0, 1
TYPES = {torch.bfloat16: BF16, torch.float32: F32}
PAIRS = {"halves": 0, "neighbours": 1}
ACTS = {"silu": 0, "gelu": 1}
CODE_BLOCK = 256  # units of one (lo, hi) pair

EXPORTS = ("gs_norm_rotate_fwd", "gs_norm_rotate_workspace_bytes", "gs_norm_rotate_bwd", "gs_cross_attn_fwd_workspace_bytes",
           "gs_cross_attn_fwd", "gs_cross_attn_bwd_workspace_bytes", "gs_cross_attn_bwd", "gs_gate8_fwd", "gs_gate8_bwd",
           "gs_layer_norm_fwd", "gs_layer_norm_workspace_bytes", "gs_layer_norm_bwd", "gs_group_mm_fwd_workspace_bytes",
           "gs_group_mm_fwd", "gs_group_mm_bwd_workspace_bytes", "gs_group_mm_bwd", "gs_adamw", "gs_adamw_moments")


class GsHeads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("batch_stride", C.c_int64), ("token_stride", C.c_int64),
                ("head_stride", C.c_int64)]


class GsNormRotate(C.Structure):
    _fields_ = [("batch", C.c_int64), ("q_len", C.c_int64), ("k_len", C.c_int64), ("q_heads", C.c_int32),
                ("k_heads", C.c_int32), ("head_dim", C.c_int32), ("rot_dim", C.c_int32), ("pairs", C.c_int32),
                ("type", C.c_int32), ("eps", C.c_float), ("n_pos", C.c_int64)]


class GsCrossAttn(C.Structure):
    _fields_ = [("batch", C.c_int64), ("q_len", C.c_int64), ("k_len", C.c_int64), ("q_heads", C.c_int32),
                ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("type", C.c_int32), ("scale", C.c_float),
                ("ranges", C.c_void_p), ("ranges_batch_stride", C.c_int64), ("ranges_row_stride", C.c_int64),
                ("key_mask", C.c_void_p), ("key_mask_batch_stride", C.c_int64)]


class GsWeights(C.Structure):
    _fields_ = [("data", C.c_void_p), ("group_stride", C.c_int64), ("k_stride", C.c_int64), ("n_stride", C.c_int64)]


class GsGroupMM(C.Structure):
    _fields_ = [("rows", C.c_int64), ("k", C.c_int64), ("n", C.c_int64), ("groups", C.c_int32), ("type", C.c_int32),
                ("offsets", C.c_void_p)]


class GsAdamWTensor(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("copy", C.c_void_p), ("n", C.c_int64), ("decay", C.c_double)]


class GsAdamWParams(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_double), ("step", C.c_int64)]


_lib = None


def lib():
    """The library, with the token operators' signatures."""
    global _lib
    if _lib is None:
        L = raster.lib()
        vp, i64, i32, sz, H = C.c_void_p, C.c_int64, C.c_int32, C.c_size_t, GsHeads
        N, A = C.POINTER(GsNormRotate), C.POINTER(GsCrossAttn)
        L.gs_norm_rotate_fwd.argtypes = [N, H, H, vp, vp, vp, vp, vp, vp, H, H, vp]
        L.gs_norm_rotate_workspace_bytes.argtypes = [N]
        L.gs_norm_rotate_bwd.argtypes = [N, H, H, H, H, vp, vp, vp, vp, vp, vp, H, H, vp, vp, vp, sz, vp]
        L.gs_cross_attn_fwd_workspace_bytes.argtypes = [A]
        L.gs_cross_attn_fwd.argtypes = [A, H, H, H, H, vp, vp, sz, vp]
        L.gs_cross_attn_bwd_workspace_bytes.argtypes = [A]
        L.gs_cross_attn_bwd.argtypes = [A, H, H, H, H, H, vp, H, H, H, vp, sz, vp]
        L.gs_gate8_fwd.argtypes = [i64, i64, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp]
        L.gs_gate8_bwd.argtypes = [i64, i64, i32, i32, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp]
        f32, W, G = C.c_float, GsWeights, C.POINTER(GsGroupMM)
        L.gs_layer_norm_fwd.argtypes = [i64, i64, i32, f32, vp, i64, vp, vp, vp, i64, vp]
        L.gs_layer_norm_workspace_bytes.argtypes = [i64, i64]
        L.gs_layer_norm_bwd.argtypes = [i64, i64, i32, f32, vp, i64, vp, i64, vp, vp, i64, vp, vp, vp, sz, vp]
        L.gs_group_mm_fwd_workspace_bytes.argtypes = [G]
        L.gs_group_mm_fwd.argtypes = [G, vp, i64, W, vp, i64, vp, sz, vp]
        L.gs_group_mm_bwd_workspace_bytes.argtypes = [G]
        L.gs_group_mm_bwd.argtypes = [G, vp, i64, vp, i64, W, vp, i64, W, vp, sz, vp]
        L.gs_adamw.argtypes = [i32, vp, i32, i32, vp, vp, vp, C.POINTER(GsAdamWParams), vp, vp]
        L.gs_adamw_moments.argtypes = [i64, vp, vp, vp, vp, vp, vp]
        for name in EXPORTS:
            getattr(L, name).restype = sz if name.endswith("_bytes") else i32
        _lib = L
    return _lib


# The smallest calls are bound by the host, so the checks are few and plain: no generators, no
# tuples made, the current stream's handle without a Stream object.


def _ptr(t):
    return None if t is None else t.data_ptr()


def _refuse(what):
    raise ValueError(what)


def _launch(name, t, *args):
    """The C call on the current stream of t's GPU, with that GPU as the current one: a default stream's work goes to
    whichever is."""
    call, at = getattr(lib(), name), t.get_device()
    if at == torch._C._cuda_getDevice():
        status = call(*args, torch._C._cuda_getCurrentRawStream(at))
    else:
        with torch.cuda.device(at):
            status = call(*args, torch._C._cuda_getCurrentRawStream(at))
    _check(status, name)


def _on(stream, call, first, *args):
    """The call with `stream` as the current one, so that what it allocates belongs to the work."""
    if stream.device_index != first.get_device():
        _refuse("a stream of the vectors' GPU")
    with torch.cuda.stream(stream):
        return call(first, *args)


def _heads(t) -> GsHeads:
    b, n, h, d = t.stride()
    if d != 1 and t.shape[3] > 1:
        _refuse("the last axis must be dense")
    return GsHeads(t.data_ptr(), b, n, h)


def _type(t) -> int:
    ty = TYPES.get(t.dtype)
    if ty is None:
        _refuse(f"bfloat16 or float32, not {t.dtype}")
    if not t.is_cuda:
        _refuse("tensors on the GPU")
    return ty


def _same(t, x, shape):
    """x has t's type, is on its GPU and has this shape."""
    if x.dtype != t.dtype or x.get_device() != t.get_device():
        _refuse("one type and one GPU for all of a call's vectors")
    if x.shape != shape:
        _refuse(f"a tensor of shape {tuple(x.shape)} in the place of one of {tuple(shape)}")


def _floats(x, shape, t, what):
    if x.dtype != torch.float32 or x.shape != shape or not x.is_contiguous() or x.get_device() != t.get_device():
        _refuse(f"{what}: float32 {tuple(shape)}, contiguous, on the vectors' GPU")


def _workspace(given, need, t):
    if given is not None:
        if not given.is_contiguous() or given.get_device() != t.get_device():
            _refuse("workspace: contiguous, on the vectors' GPU")
        return given, given.numel() * given.element_size()
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=t.device), need


# -- norm with rotation ----------------------------------------------------------------------


def _norm_shape(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs) -> GsNormRotate:
    if q.dim() != 4 or k.dim() != 4:
        _refuse("q [batch][tokens][heads][d], k [batch][keys][heads][d]")
    B, Lq, Hq, D = q.shape
    _, Lk, Hk, _ = k.shape
    if pairs not in PAIRS:
        _refuse(f"pairs: one of {tuple(PAIRS)}")
    ty = _type(q)
    _same(q, k, (B, Lk, Hk, D))
    _floats(wq, (D,), q, "wq")
    _floats(wk, (D,), q, "wk")
    if cos.dim() != 2:
        _refuse("cos, sin: [positions][pairs]")
    n, half = cos.shape
    _floats(cos, (n, half), q, "cos")
    _floats(sin, (n, half), q, "sin")
    for pos, length in ((pos_q, Lq), (pos_k, Lk)):
        if pos is not None and (pos.dtype != torch.int32 or pos.shape != (B, length) or not pos.is_contiguous()
                                or pos.get_device() != q.get_device()):
            _refuse("positions: int32 [batch][tokens], contiguous, on the vectors' GPU")
    return GsNormRotate(B, Lq, Lk, Hq, Hk, D, 2 * half, PAIRS[pairs], ty, eps, n)


def norm_rotate_fwd(q, k, wq, wk, cos, sin, pos_q=None, pos_k=None, eps: float = 1e-6, pairs: str = "halves",
                    out: tuple | None = None, stream=None) -> tuple:
    """gs_norm_rotate_fwd: (q, k) normed by head, weighted and rotated.  q [B, Lq, Hq, D],
    k [B, Lk, Hk, D]; cos, sin [positions, pairs]; ``out``: the two outputs' tensors (may be q, k)."""
    if stream is not None:
        return _on(stream, norm_rotate_fwd, q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs, out)
    p = _norm_shape(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)
    if out is None:
        oq, ok = torch.empty_like(q), torch.empty_like(k)
    else:
        oq, ok = out
        _same(q, oq, q.shape)
        _same(q, ok, k.shape)
    _launch("gs_norm_rotate_fwd", q, p, _heads(q), _heads(k), wq.data_ptr(), wk.data_ptr(), cos.data_ptr(), sin.data_ptr(),
            _ptr(pos_q), _ptr(pos_k), _heads(oq), _heads(ok))
    return oq, ok


def norm_rotate_bwd(dout_q, dout_k, q, k, wq, wk, cos, sin, pos_q=None, pos_k=None, eps: float = 1e-6,
                    pairs: str = "halves", workspace=None, stream=None) -> tuple:
    """gs_norm_rotate_bwd: (dq, dk, dwq, dwk) from the inputs of the forward call and its outputs' gradients."""
    if stream is not None:
        return _on(stream, norm_rotate_bwd, dout_q, dout_k, q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs, workspace)
    p = _norm_shape(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)
    _same(q, dout_q, q.shape)
    _same(q, dout_k, k.shape)
    L = lib()
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dwq, dwk = torch.empty_like(wq), torch.empty_like(wk)
    ws, n = _workspace(workspace, L.gs_norm_rotate_workspace_bytes(p), q)
    _launch("gs_norm_rotate_bwd", q, p, _heads(dout_q), _heads(dout_k), _heads(q), _heads(k), wq.data_ptr(), wk.data_ptr(),
            cos.data_ptr(), sin.data_ptr(), _ptr(pos_q), _ptr(pos_k), _heads(dq), _heads(dk),
            dwq.data_ptr(), dwk.data_ptr(), _ptr(ws), n)
    return dq, dk, dwq, dwk


# -- cross attention -------------------------------------------------------------------------


def _attn_shape(q, k, v, scale, ranges, key_mask) -> GsCrossAttn:
    if q.dim() != 4 or k.dim() != 4:
        _refuse("q [batch][rows][heads][d]; k and v [batch][keys][kv heads][d]")
    B, Lq, Hq, D = q.shape
    _, Lk, Hk, _ = k.shape
    ty = _type(q)
    _same(q, k, (B, Lk, Hk, D))
    _same(q, v, (B, Lk, Hk, D))
    p = GsCrossAttn(B, Lq, Lk, Hq, Hk, D, ty, D**-0.5 if scale is None else scale)
    if ranges is not None:
        if (ranges.dtype != torch.int32 or ranges.get_device() != q.get_device() or ranges.dim() != 3
                or ranges.shape[0] not in (1, B) or ranges.shape[1] not in (1, Lq) or ranges.shape[2] != 2
                or (ranges.numel() and (ranges.stride(2) != 1 or ranges.stride(0) % 2 or ranges.stride(1) % 2))):
            _refuse("ranges: int32 [batch or 1][rows or 1][2], pairs dense, on the vectors' GPU")
        p.ranges = ranges.data_ptr()
        p.ranges_batch_stride = ranges.stride(0) // 2 if ranges.shape[0] > 1 else 0
        p.ranges_row_stride = ranges.stride(1) // 2 if ranges.shape[1] > 1 else 0
    if key_mask is not None:
        if (key_mask.dtype not in (torch.uint8, torch.bool) or key_mask.get_device() != q.get_device()
                or key_mask.dim() != 2 or key_mask.shape[0] not in (1, B) or key_mask.shape[1] != Lk
                or (Lk > 1 and key_mask.stride(1) != 1)):
            _refuse("key_mask: bytes or truth values [batch or 1][keys], on the vectors' GPU")
        p.key_mask = key_mask.data_ptr()
        p.key_mask_batch_stride = key_mask.stride(0) if key_mask.shape[0] > 1 else 0
    return p


def cross_attn_fwd(q, k, v, scale: float | None = None, ranges=None, key_mask=None, out=None, lse=None, workspace=None,
                   stream=None) -> tuple:
    """gs_cross_attn_fwd: (out, lse).  q [B, Lq, Hq, D], k and v [B, Lk, Hk, D]; ``ranges`` [B or 1, Lq or 1, 2]: the
    keys [first, last) of each row (one row: lengths of sequences); ``key_mask`` [B or 1, Lk]: 0 hides a key; ``scale``
    None: 1 / sqrt(D)."""
    if stream is not None:
        return _on(stream, cross_attn_fwd, q, k, v, scale, ranges, key_mask, out, lse, workspace)
    p = _attn_shape(q, k, v, scale, ranges, key_mask)
    shape = (p.batch, p.q_heads, p.q_len)
    if out is None:
        out = torch.empty_like(q)
    else:
        _same(q, out, q.shape)
    if lse is None:
        lse = torch.empty(shape, dtype=torch.float32, device=q.device)
    else:
        _floats(lse, shape, q, "lse")
    L = lib()
    ws, n = _workspace(workspace, L.gs_cross_attn_fwd_workspace_bytes(p), q)
    _launch("gs_cross_attn_fwd", q, p, _heads(q), _heads(k), _heads(v), _heads(out), lse.data_ptr(), _ptr(ws), n)
    return out, lse


def cross_attn_bwd(dout, q, k, v, out, lse, scale: float | None = None, ranges=None, key_mask=None, workspace=None,
                   stream=None) -> tuple:
    """gs_cross_attn_bwd: (dq, dk, dv) from the forward call's inputs and outputs and the gradient of out."""
    if stream is not None:
        return _on(stream, cross_attn_bwd, dout, q, k, v, out, lse, scale, ranges, key_mask, workspace)
    p = _attn_shape(q, k, v, scale, ranges, key_mask)
    _same(q, dout, q.shape)
    _same(q, out, q.shape)
    _floats(lse, (p.batch, p.q_heads, p.q_len), q, "lse")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    L = lib()
    ws, n = _workspace(workspace, L.gs_cross_attn_bwd_workspace_bytes(p), q)
    _launch("gs_cross_attn_bwd", q, p, _heads(dout), _heads(q), _heads(k), _heads(v), _heads(out), lse.data_ptr(), _heads(dq),
            _heads(dk), _heads(dv), _ptr(ws), n)
    return dq, dk, dv


# -- gated activation with 8-bit checkpoints -------------------------------------------------


def _stride(x, t, rows, width):
    """x's row stride; it is a matrix [rows][width] of t's type on its GPU, its rows dense."""
    _same(t, x, (rows, width))
    if width > 1 and x.stride(1) != 1:
        _refuse("matrices [rows][width], rows dense")
    return x.stride(0)


def gate8_fwd(gate, up, act: str = "silu", stream=None) -> tuple:
    """gs_gate8_fwd: (y, codes, bounds) of act(gate) * up; gate, up [rows, width] (views of one projection's output
    are taken as they are).  codes uint8 [2, rows, width] and bounds float32 [2, rows, blocks, 2] are what
    gate8_bwd needs."""
    if stream is not None:
        return _on(stream, gate8_fwd, gate, up, act)
    if act not in ACTS:
        _refuse(f"act: one of {tuple(ACTS)}")
    if gate.dim() != 2:
        _refuse("matrices [rows][width]")
    ty = _type(gate)
    rows, width = gate.shape
    gs, us = _stride(gate, gate, rows, width), _stride(up, gate, rows, width)
    dev = gate.device
    y = torch.empty_like(gate)
    codes = torch.empty((2, rows, width), dtype=torch.uint8, device=dev)
    bounds = torch.empty((2, rows, (width + CODE_BLOCK - 1) // CODE_BLOCK, 2), dtype=torch.float32, device=dev)
    _launch("gs_gate8_fwd", gate, rows, width, ACTS[act], ty, gate.data_ptr(), gs, up.data_ptr(), us, y.data_ptr(), y.stride(0),
            codes.data_ptr(), bounds.data_ptr())
    return y, codes, bounds


def gate8_bwd(dy, codes, bounds, act: str = "silu", with_y: bool = True, dgate=None, dup=None, stream=None) -> tuple:
    """gs_gate8_bwd: (dgate, dup, y again or None) from the codes; ``dgate``, ``dup``: tensors to write to, such as the
    halves of one [rows, 2 * width] gradient."""
    if stream is not None:
        return _on(stream, gate8_bwd, dy, codes, bounds, act, with_y, dgate, dup)
    if act not in ACTS:
        _refuse(f"act: one of {tuple(ACTS)}")
    if dy.dim() != 2:
        _refuse("matrices [rows][width]")
    ty = _type(dy)
    rows, width = dy.shape
    if codes.dtype != torch.uint8 or codes.shape != (2, rows, width) or not codes.is_contiguous() or codes.get_device() != dy.get_device():
        _refuse("codes: gate8_fwd's")
    _floats(bounds, (2, rows, (width + CODE_BLOCK - 1) // CODE_BLOCK, 2), dy, "bounds")
    ds = _stride(dy, dy, rows, width)
    dgate = torch.empty_like(dy) if dgate is None else dgate
    dup = torch.empty_like(dy) if dup is None else dup
    y = torch.empty_like(dy) if with_y else None
    _launch("gs_gate8_bwd", dy, rows, width, ACTS[act], ty, dy.data_ptr(), ds, codes.data_ptr(), bounds.data_ptr(),
            dgate.data_ptr(), _stride(dgate, dy, rows, width), dup.data_ptr(), _stride(dup, dy, rows, width),
            _ptr(y), y.stride(0) if with_y else 0)
    return dgate, dup, y


# -- layer norm ------------------------------------------------------------------------------


def _new(x, rows, width):
    """A dense matrix of x's type on its GPU (the shortest of torch's ways to make one: 1.3 us, or 1.6)."""
    return torch.empty_like(x) if x.shape == (rows, width) and x.is_contiguous() else x.new_empty((rows, width))


def _matrix(x):
    if x.dim() != 2:
        _refuse("matrices [rows][width]")
    return x.shape


def layer_norm_fwd(x, w=None, b=None, eps: float = 1e-5, out=None, stream=None):
    """gs_layer_norm_fwd: rows of x [rows, width] with mean 0 and variance 1, times w, plus b (float32 [width]; None: 1
    and 0).  ``out``: a tensor to write to (may be x)."""
    if stream is not None:
        return _on(stream, layer_norm_fwd, x, w, b, eps, out)
    rows, width = _matrix(x)
    ty = _type(x)
    xs = _stride(x, x, rows, width)
    if w is not None:
        _floats(w, (width,), x, "w")
    if b is not None:
        _floats(b, (width,), x, "b")
    if out is None:
        out = _new(x, rows, width)
    _launch("gs_layer_norm_fwd", x, rows, width, ty, eps, x.data_ptr(), xs, _ptr(w), _ptr(b), out.data_ptr(), _stride(out, x, rows, width))
    return out


def layer_norm_bwd(dy, x, w=None, eps: float = 1e-5, with_dw: bool = True, with_db: bool = True, dx=None, workspace=None,
                   stream=None) -> tuple:
    """gs_layer_norm_bwd: (dx, dw or None, db or None) from the forward call's inputs and the gradient of its result;
    ``dx``: a tensor to write to (may be dy or x)."""
    if stream is not None:
        return _on(stream, layer_norm_bwd, dy, x, w, eps, with_dw, with_db, dx, workspace)
    rows, width = _matrix(x)
    ty = _type(x)
    xs, ds = _stride(x, x, rows, width), _stride(dy, x, rows, width)
    if w is not None:
        _floats(w, (width,), x, "w")
    if dx is None:
        dx = _new(x, rows, width)
    dw = torch.empty(width, dtype=torch.float32, device=x.device) if with_dw else None
    db = torch.empty(width, dtype=torch.float32, device=x.device) if with_db else None
    ws, n = _workspace(workspace, lib().gs_layer_norm_workspace_bytes(rows, width) if with_dw or with_db else 0, x)
    _launch("gs_layer_norm_bwd", x, rows, width, ty, eps, dy.data_ptr(), ds, x.data_ptr(), xs, _ptr(w), dx.data_ptr(),
            _stride(dx, x, rows, width), _ptr(dw), _ptr(db), _ptr(ws), n)
    return dx, dw, db


# -- products grouped by rows ----------------------------------------------------------------


def _weights(w, x, k, of=None) -> GsWeights:
    """Weights for rows of k units; ``of``: the weights that these are the gradients of."""
    if w.dim() != 3:
        _refuse("weights [groups][k][n]")
    _same(x, w, (w.shape[0], k, w.shape[2]) if of is None else of.shape)
    g, i, j = w.stride()
    if j != 1 and i != 1 and w.shape[1] > 1 and w.shape[2] > 1:
        _refuse("weights with one of their last two axes dense")
    return GsWeights(w.data_ptr(), g, i, j)


def _group_shape(x, w, offsets) -> tuple:
    rows, k = _matrix(x)
    ty = _type(x)
    ww = _weights(w, x, k)
    groups, _, n = w.shape
    if (offsets.dtype != torch.int32 or offsets.shape != (groups + 1,) or not offsets.is_contiguous()
            or offsets.get_device() != x.get_device()):
        _refuse("offsets: int32 [groups + 1], contiguous, on the vectors' GPU")
    return GsGroupMM(rows, k, n, groups, ty, offsets.data_ptr()), ww


def group_mm_fwd(x, w, offsets, out=None, workspace=None, stream=None):
    """gs_group_mm_fwd: every row of x [rows, k] times its group's weights, y [rows, n].  w [groups, k, n], either of its
    last two axes dense (a linear layer's weights [groups, n, k] transposed); offsets int32 [groups + 1] on the GPU: group
    g has the rows from offsets[g] to offsets[g + 1].  Rows of no group get 0.  ``out``: a tensor to write to, apart from the inputs."""
    if stream is not None:
        return _on(stream, group_mm_fwd, x, w, offsets, out, workspace)
    p, ww = _group_shape(x, w, offsets)
    if out is None:
        out = _new(x, p.rows, p.n)
    ws, n = _workspace(workspace, lib().gs_group_mm_fwd_workspace_bytes(p), x)
    _launch("gs_group_mm_fwd", x, p, x.data_ptr(), _stride(x, x, p.rows, p.k), ww, out.data_ptr(), _stride(out, x, p.rows, p.n),
            _ptr(ws), n)
    return out


def group_mm_bwd(dy, x, w, offsets, with_dx: bool = True, with_dw: bool = True, dx=None, dw=None, workspace=None,
                 stream=None) -> tuple:
    """gs_group_mm_bwd: (dx or None, dw or None) from the forward call's inputs and the gradient of its result; ``dx``,
    ``dw``: tensors to write to, apart from the inputs and each other (dw lies as w does where it is not given)."""
    if stream is not None:
        return _on(stream, group_mm_bwd, dy, x, w, offsets, with_dx, with_dw, dx, dw, workspace)
    p, ww = _group_shape(x, w, offsets)
    ds = _stride(dy, x, p.rows, p.n)
    if not with_dx:
        dx = None
    elif dx is None:
        dx = _new(x, p.rows, p.k)
    if not with_dw:
        dw = None
    elif dw is None:
        dw = torch.empty_like(w)
    ws, n = _workspace(workspace, lib().gs_group_mm_bwd_workspace_bytes(p), x)
    _launch("gs_group_mm_bwd", x, p, dy.data_ptr(), ds, x.data_ptr(), _stride(x, x, p.rows, p.k), ww, _ptr(dx),
            0 if dx is None else _stride(dx, x, p.rows, p.k), GsWeights() if dw is None else _weights(dw, x, p.k, w),
            _ptr(ws), n)
    return dx, dw


# -- AdamW over many tensors -----------------------------------------------------------------


_dtype, _F32 = operator.attrgetter("dtype"), (torch.float32,)


class AdamWState:
    """Moments of a list of tensors, one after another, each from a multiple of 256 units on: float32 (bounds None), or
    int8 and uint8 codes with bounds float32 [blocks, 2]."""

    __slots__ = ("m", "v", "bounds")

    def __init__(self, m, v, bounds=None):
        self.m, self.v, self.bounds = m, v, bounds


def _blocks(tensors) -> int:
    return sum([(t.numel() + CODE_BLOCK - 1) // CODE_BLOCK for t in tensors])


def adamw_state(params, bits: int = 8) -> AdamWState:
    """Zero moments for ``params``, in 8 bits or in 32.  In 8 bits a moment decays by whole codes only: beside a unit that keeps the
    bound of its 256 up, small first moments and (with a beta2 past 0.992) all second ones stay as they are while their gradients are
    0, so tensors whose neighbouring units fare differently for long want 32."""
    if bits not in (8, 32):
        _refuse("bits: 8 or 32")
    if not params:
        _refuse("a list of tensors")
    blocks, dev = _blocks(params), params[0].device
    if bits == 32:
        return AdamWState(torch.zeros(blocks * CODE_BLOCK, device=dev), torch.zeros(blocks * CODE_BLOCK, device=dev))
    return AdamWState(torch.zeros(blocks * CODE_BLOCK, dtype=torch.int8, device=dev), torch.zeros(blocks * CODE_BLOCK, dtype=torch.uint8, device=dev),
                      torch.zeros((blocks, 2), device=dev))


def _state_bits(state, blocks: int, dev: int) -> int:
    m, v, bounds = state.m, state.v, state.bounds
    bits = 32 if bounds is None else 8
    for x, types in ((m, (torch.float32, torch.int8)), (v, (torch.float32, torch.uint8))):
        if x.dtype != types[bits == 8] or x.shape != (blocks * CODE_BLOCK,) or not x.is_contiguous() or x.get_device() != dev:
            _refuse("state: adamw_state's of these tensors")
    if bits == 8 and (bounds.dtype != torch.float32 or bounds.shape != (blocks, 2) or not bounds.is_contiguous() or bounds.get_device() != dev):
        _refuse("state: adamw_state's of these tensors")
    return bits


def adamw(params, grads, state: AdamWState, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
          weight_decay=0.0, copies=None, grad_scale=None, stream=None) -> None:
    """gs_adamw: one step over lists of tensors, params (float32) and state in place.  grads: all float32 or all bfloat16, of the
    params' sizes; ``weight_decay``: a number, or one for each tensor; ``copies``: bfloat16 tensors (or None) that receive
    the new parameters; ``grad_scale``: a float32 tensor of one element that multiplies the gradients.  Every tensor is
    contiguous and no two of params and copies overlap."""
    if stream is not None:
        return _on(stream, lambda first: adamw(params, grads, state, lr, step, beta1, beta2, eps, weight_decay, copies, grad_scale), state.m)
    count, dev = len(params), state.m.get_device()
    if len(grads) != count or (copies is not None and len(copies) != count):
        _refuse("a gradient (and a copy) for each tensor")
    if not state.m.is_cuda:
        _refuse("tensors on the GPU")
    # a check of all tensors at a time: a third of what a loop over them takes
    size, dense, device, pointer = torch.Tensor.numel, torch.Tensor.is_contiguous, torch.Tensor.get_device, torch.Tensor.data_ptr
    try:
        sizes, types = list(map(size, params)), set(map(_dtype, grads))
        if list(map(size, grads)) != sizes or not types.issubset(TYPES) or len(types) > 1 or not set(map(_dtype, params)).issubset(_F32):
            _refuse("params float32, gradients all float32 or all bfloat16 and of the params' sizes")
    except (TypeError, AttributeError):
        _refuse("tensors: a gradient for each (None is none)")
    if not (all(map(dense, params)) and all(map(dense, grads))):
        _refuse("params and gradients, all contiguous")
    if not set(map(device, params)).union(map(device, grads)).issubset((dev,)):
        _refuse("one GPU for all of a call's tensors")
    ty = TYPES[types.pop()] if count else TYPES[torch.float32]
    at, pointers, to = list(map(pointer, params)), list(map(pointer, grads)), [0] * count
    if copies is not None:
        where = [i for i, c in enumerate(copies) if c is not None]
        given = [copies[i] for i in where]
        if (list(map(size, given)) != [sizes[i] for i in where] or not set(map(_dtype, given)).issubset((torch.bfloat16,)) or not all(map(dense, given))
                or not set(map(device, given)).issubset((dev,))):
            _refuse("copies: bfloat16, of the params' sizes, contiguous, on the params' GPU")
        for i, c in zip(where, map(pointer, given)):
            to[i] = c
    written = list(filter(None, at if copies is None else at + to))
    if 0 in sizes:
        written = [a for a, n in zip(at + to, sizes + sizes) if a and n]
    if len(set(written)) != len(written):
        _refuse("a tensor is given twice")
    bits = _state_bits(state, sum([(n + CODE_BLOCK - 1) // CODE_BLOCK for n in sizes]), dev)
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.get_device() != dev):
        _refuse("grad_scale: one float32 on the params' GPU")
    if isinstance(weight_decay, (int, float)):
        decay = [struct.unpack("=q", struct.pack("=d", weight_decay))[0]] * count
    elif len(weight_decay) != count:
        _refuse("weight_decay: a number, or one for each tensor")
    else:
        decay = struct.unpack(f"={count}q", struct.pack(f"={count}d", *weight_decay))
    # GsAdamWTensor[count], a column at a time
    table = array("q", bytes(C.sizeof(GsAdamWTensor) * count))
    for i, column in enumerate((at, pointers, to, sizes, decay)):
        table[i::5] = array("q", column)
    _launch("gs_adamw", state.m, count, table.buffer_info()[0], ty, bits, state.m.data_ptr(), state.v.data_ptr(), _ptr(state.bounds),
            GsAdamWParams(lr, beta1, beta2, eps, int(step)), _ptr(grad_scale))
    # what torch saved of these tensors for a backward pass is no longer what it saved
    torch.autograd.graph.increment_version(params)
    if copies is not None:
        torch.autograd.graph.increment_version(given)


def adamw_moments(state: AdamWState, stream=None) -> tuple:
    """(m, v) float32 as the state holds them: what its codes stand for, or its own tensors."""
    if stream is not None:
        return _on(stream, lambda first: adamw_moments(state), state.m)
    if state.bounds is None:
        return state.m, state.v
    blocks = state.bounds.shape[0]
    if not state.m.is_cuda:
        _refuse("tensors on the GPU")
    _state_bits(state, blocks, state.m.get_device())
    m = torch.empty(blocks * CODE_BLOCK, dtype=torch.float32, device=state.m.device)
    v = torch.empty_like(m)
    _launch("gs_adamw_moments", state.m, blocks, state.m.data_ptr(), state.v.data_ptr(), state.bounds.data_ptr(), m.data_ptr(), v.data_ptr())
    return m, v


# -- as differentiable torch functions -------------------------------------------------------


def _on_vectors(t):
    """t itself where the C calls take it as it is, a dense copy where they do not (an expanded gradient, or one that starts off 16 bytes)."""
    each = 16 // t.element_size()
    dense = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s % each == 0 or n == 1 for s, n in zip(t.stride()[:-1], t.shape))
    return t if dense else t.clone(memory_format=torch.contiguous_format)  # (contiguous() keeps one that is only off its boundary)


class _Linked(torch.autograd.Function):
    """The first n tensors as they are, with every other one as a source that cannot be differentiated for."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of the library's calls can be differentiated once only")


def once(backward):
    """Marks a backward pass whose gradients torch did not record.  Where they are to be differentiated again
    (create_graph), they are linked to all that they come from (the outputs' gradients and what forward saved), so
    that a second derivative on any such path is an error and not a sum without this part."""

    @functools.wraps(backward)
    def run(ctx, *douts):
        if not torch.is_grad_enabled():
            return backward(ctx, *douts)
        with torch.no_grad():
            grads = backward(ctx, *douts)
        made = [g for g in grads if g is not None]
        linked = iter(_Linked.apply(len(made), *made, *douts, *ctx.saved_tensors))
        return tuple(None if g is None else next(linked) for g in grads)

    return run


class _NormRotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, pos_q, pos_k)
        ctx.more = (eps, pairs)
        return norm_rotate_fwd(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)

    @staticmethod
    @once
    def backward(ctx, dq, dk):
        return (*norm_rotate_bwd(_on_vectors(dq), _on_vectors(dk), *ctx.saved_tensors, *ctx.more), *([None] * 6))


def norm_rotate(q, k, wq, wk, cos, sin, pos_q=None, pos_k=None, eps: float = 1e-6, pairs: str = "halves") -> tuple:
    """norm_rotate_fwd with gradients for q, k, wq and wk."""
    return _NormRotate.apply(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)


class _CrossAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale, ranges, key_mask):
        out, lse = cross_attn_fwd(q, k, v, scale, ranges, key_mask)
        ctx.save_for_backward(q, k, v, out, lse, ranges, key_mask)
        ctx.scale = scale
        return out

    @staticmethod
    @once
    def backward(ctx, dout):
        q, k, v, out, lse, ranges, key_mask = ctx.saved_tensors
        return (*cross_attn_bwd(_on_vectors(dout), q, k, v, out, lse, ctx.scale, ranges, key_mask), None, None, None)


def cross_attention(q, k, v, scale: float | None = None, ranges=None, key_mask=None):
    """cross_attn_fwd's out with gradients for q, k and v."""
    return _CrossAttention.apply(q, k, v, scale, ranges, key_mask)


class _Gated8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, act):
        width = h.shape[-1] // 2
        flat = h.reshape(math.prod(h.shape[:-1]), 2 * width)
        y, codes, bounds = gate8_fwd(flat[:, :width], flat[:, width:], act)
        link = h.new_empty(0)  # h's place in the graph, without h
        ctx.save_for_backward(codes, bounds, link)
        ctx.act, ctx.shape = act, h.shape
        return y.view(*h.shape[:-1], width), link

    @staticmethod
    @once
    def backward(ctx, dy, _):
        codes, bounds, _ = ctx.saved_tensors
        width = codes.shape[2]
        dh = torch.empty((codes.shape[1], 2 * width), dtype=dy.dtype, device=dy.device)
        dy = dy.reshape(codes.shape[1], width)
        dy = dy if dy.stride() == (width, 1) else dy.contiguous()
        gate8_bwd(dy, codes, bounds, ctx.act, False, dh[:, :width], dh[:, width:])
        return dh.view(ctx.shape), None


def gated8(h, act: str = "silu"):
    """act(gate) * up of a projection's output h [..., 2 * width] = (gate | up), with the gradient for h from 8-bit
    codes: between the passes this keeps the codes and their bounds, a quarter (float32) or half (bfloat16) of h.  (A
    product that follows keeps its own input; gate8_bwd makes it again where a backward pass is written by hand.)"""
    if h.dim() == 0 or h.shape[-1] % 2:
        _refuse("a last axis of two halves, gate and up")
    return _Gated8.apply(h, act)[0]


def _rows(t, width):
    """t as a matrix [rows][width] with dense rows that do not overlap, as it is where it can be."""
    t = t.reshape(math.prod(t.shape[:-1]), width)
    dense = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    return t if dense else t.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, eps):
        ctx.save_for_backward(x, w)  # x itself: a view of it would hide from torch what is changed in between
        ctx.eps = eps
        return layer_norm_fwd(_rows(x, x.shape[-1]), w, b, eps).view(x.shape)

    @staticmethod
    @once
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        width = x.shape[-1]
        dx, dw, db = layer_norm_bwd(_rows(dy, width), _rows(x, width), w, ctx.eps, ctx.needs_input_grad[1], ctx.needs_input_grad[2])
        return dx.view(x.shape), dw, db, None


def layer_norm(x, w=None, b=None, eps: float = 1e-5):
    """layer_norm_fwd over the last axis of x [..., width], with gradients for x, w and b."""
    if x.dim() == 0:
        _refuse("a last axis to norm over")
    return _LayerNorm.apply(x, w, b, eps)


def _dense(x):
    """The matrix x as it is, or a copy where its rows are not dense."""
    return x if _matrix(x)[1] <= 1 or x.stride(1) == 1 else x.contiguous()


class _GroupMM(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)  # x itself, as _LayerNorm has it
        return group_mm_fwd(_dense(x), w, offsets)

    @staticmethod
    @once
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        return (*group_mm_bwd(_rows(dy, w.shape[2]), _dense(x), w, offsets, ctx.needs_input_grad[0], ctx.needs_input_grad[1]), None)


def group_mm(x, w, offsets):
    """group_mm_fwd with gradients for x and w; an x whose rows are not dense is copied."""
    return _GroupMM.apply(x, w, offsets)
