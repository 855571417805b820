"""ctypes binding of libgsraster's token operators (the C ABI in include/gs_tokens.h).

The parts of a decoder layer that predicts Gaussians from images which are not plain matrix
products: norms of queries and keys with the position rotation, attention of the tokens to the
encoder's states, and the gated activation that keeps its inputs as 8-bit codes.

Tensors are bfloat16 or float32 on the GPU, laid out as include/gs_tokens.h says: vectors dense in
their last axis, on 16-byte boundaries, any strides else (views of one projection's output are
taken as they are).  Shapes and types are checked here (the C calls do not see them: ValueError),
everything else by the C calls (raster.GsError).  Work goes to the current stream, or to
``stream``; outputs and workspaces are torch tensors made on the calling stream unless given.

``norm_rotate``, ``cross_attention`` and ``gated8`` are the same operators as differentiable
torch functions.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import raster
from .raster import _check, _stream

BF16, F32 = 0, 1
TYPES = {torch.bfloat16: BF16, torch.float32: F32}
PAIRS = {"halves": 0, "neighbours": 1}
ACTS = {"silu": 0, "gelu": 1}
CODE_BLOCK = 256  # units of one (lo, hi) pair

EXPORTS = ("gs_norm_rotate_fwd", "gs_norm_rotate_workspace_bytes", "gs_norm_rotate_bwd", "gs_cross_attn_fwd_workspace_bytes",
           "gs_cross_attn_fwd", "gs_cross_attn_bwd_workspace_bytes", "gs_cross_attn_bwd", "gs_gate8_fwd", "gs_gate8_bwd")


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
        for name in EXPORTS:
            getattr(L, name).restype = sz if name.endswith("_bytes") else i32
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _heads(t) -> GsHeads:
    s = t.stride()
    _require(s[3] == 1 or t.shape[3] == 1, "the last axis must be dense")
    return GsHeads(t.data_ptr(), s[0], s[1], s[2])


def _type(*tensors) -> int:
    t = tensors[0].dtype
    _require(t in TYPES, f"bfloat16 or float32, not {t}")
    dev = tensors[0].device
    _require(dev.type == "cuda", "tensors on the GPU")
    for x in tensors:
        _require(x.dtype == t and x.device == dev, "one type and one device for all of a call's vectors")
    return TYPES[t]


def _floats(t, shape, what):
    _require(t.dtype == torch.float32 and tuple(t.shape) == shape and t.is_contiguous() and t.is_cuda,
             f"{what}: float32 {shape}, contiguous, on the GPU")


def _workspace(given, need, device):
    if given is not None:
        _require(given.is_contiguous() and given.device == device, "workspace: contiguous, on the same GPU")
        return given, given.numel() * given.element_size()
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=device), need


# -- norm with rotation ----------------------------------------------------------------------


def _norm_shape(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs) -> GsNormRotate:
    _require(q.dim() == 4 and k.dim() == 4 and q.shape[0] == k.shape[0] and q.shape[3] == k.shape[3],
             "q [batch][tokens][heads][d] and k of the same batch and d")
    _require(pairs in PAIRS, f"pairs: one of {tuple(PAIRS)}")
    B, Lq, Hq, D = q.shape
    _floats(wq, (D,), "wq")
    _floats(wk, (D,), "wk")
    _require(cos.dim() == 2, "cos, sin: [positions][pairs]")
    _floats(cos, tuple(cos.shape), "cos")
    _floats(sin, tuple(cos.shape), "sin")
    for pos, n in ((pos_q, Lq), (pos_k, k.shape[1])):
        _require(pos is None or (pos.dtype == torch.int32 and tuple(pos.shape) == (B, n) and pos.is_contiguous()
                                 and pos.is_cuda), "positions: int32 [batch][tokens], contiguous, on the GPU")
    return GsNormRotate(B, Lq, k.shape[1], Hq, k.shape[2], D, 2 * cos.shape[1], PAIRS[pairs], _type(q, k), eps,
                        cos.shape[0])


def norm_rotate_fwd(q, k, wq, wk, cos, sin, pos_q=None, pos_k=None, eps: float = 1e-6, pairs: str = "halves",
                    out: tuple | None = None, stream=None) -> tuple:
    """gs_norm_rotate_fwd: (q, k) normed by head, weighted and rotated.  q [B, Lq, Hq, D],
    k [B, Lk, Hk, D]; cos, sin [positions, pairs]; ``out``: the two outputs' tensors (may be q, k)."""
    p = _norm_shape(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device), torch.empty(k.shape, dtype=k.dtype, device=k.device))
    oq, ok = out
    _require(oq.shape == q.shape and ok.shape == k.shape, "out: the inputs' shapes")
    _type(q, oq, ok)
    _check(lib().gs_norm_rotate_fwd(p, _heads(q), _heads(k), _ptr(wq), _ptr(wk), _ptr(cos), _ptr(sin), _ptr(pos_q),
                                    _ptr(pos_k), _heads(oq), _heads(ok), _stream(stream)), "gs_norm_rotate_fwd")
    return oq, ok


def norm_rotate_bwd(dout_q, dout_k, q, k, wq, wk, cos, sin, pos_q=None, pos_k=None, eps: float = 1e-6,
                    pairs: str = "halves", workspace=None, stream=None) -> tuple:
    """gs_norm_rotate_bwd: (dq, dk, dwq, dwk) from the inputs of the forward call and its outputs' gradients."""
    p = _norm_shape(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)
    _require(dout_q.shape == q.shape and dout_k.shape == k.shape, "dout_q, dout_k: the inputs' shapes")
    _type(q, dout_q, dout_k)
    L, dev, D = lib(), q.device, q.shape[3]
    dq, dk = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=k.dtype, device=dev)
    dw = torch.empty((2, D), dtype=torch.float32, device=dev)
    dwq, dwk = dw.unbind(0)
    ws, n = _workspace(workspace, L.gs_norm_rotate_workspace_bytes(p), dev)
    _check(L.gs_norm_rotate_bwd(p, _heads(dout_q), _heads(dout_k), _heads(q), _heads(k), _ptr(wq), _ptr(wk), _ptr(cos),
                                _ptr(sin), _ptr(pos_q), _ptr(pos_k), _heads(dq), _heads(dk), _ptr(dwq), _ptr(dwk),
                                _ptr(ws), n, _stream(stream)), "gs_norm_rotate_bwd")
    return dq, dk, dwq, dwk


# -- cross attention -------------------------------------------------------------------------


def _attn_shape(q, k, v, scale, ranges, key_mask) -> GsCrossAttn:
    _require(q.dim() == 4 and k.dim() == 4 and k.shape == v.shape and q.shape[0] == k.shape[0] and q.shape[3] == k.shape[3],
             "q [batch][rows][heads][d]; k and v [batch][keys][kv heads][d]")
    B, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1], k.shape[2]
    p = GsCrossAttn(B, Lq, Lk, Hq, Hk, D, _type(q, k, v), D**-0.5 if scale is None else scale)
    if ranges is not None:
        _require(ranges.dtype == torch.int32 and ranges.is_cuda and ranges.dim() == 3 and ranges.shape[0] in (1, B)
                 and ranges.shape[1] in (1, Lq) and ranges.shape[2] == 2 and (ranges.numel() == 0 or ranges.stride(2) == 1)
                 and ranges.stride(0) % 2 == 0 and ranges.stride(1) % 2 == 0,
                 "ranges: int32 [batch or 1][rows or 1][2], pairs dense, on the GPU")
        p.ranges = ranges.data_ptr()
        p.ranges_batch_stride = ranges.stride(0) // 2 if ranges.shape[0] > 1 else 0
        p.ranges_row_stride = ranges.stride(1) // 2 if ranges.shape[1] > 1 else 0
    if key_mask is not None:
        _require(key_mask.dtype in (torch.uint8, torch.bool) and key_mask.is_cuda and tuple(key_mask.shape) in ((B, Lk), (1, Lk))
                 and (Lk <= 1 or key_mask.stride(1) == 1), "key_mask: bytes or truth values [batch or 1][keys], on the GPU")
        p.key_mask = key_mask.data_ptr()
        p.key_mask_batch_stride = key_mask.stride(0) if key_mask.shape[0] > 1 else 0
    return p


def cross_attn_fwd(q, k, v, scale: float | None = None, ranges=None, key_mask=None, out=None, lse=None, workspace=None,
                   stream=None) -> tuple:
    """gs_cross_attn_fwd: (out, lse).  q [B, Lq, Hq, D], k and v [B, Lk, Hk, D]; ``ranges`` [B or 1, Lq or 1, 2]: the
    keys [first, last) of each row (one row: lengths of sequences); ``key_mask`` [B or 1, Lk]: 0 hides a key; ``scale``
    None: 1 / sqrt(D)."""
    p = _attn_shape(q, k, v, scale, ranges, key_mask)
    dev = q.device
    B, Lq, Hq, _ = q.shape
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=dev)
    _require(out.shape == q.shape, "out: q's shape")
    _type(q, out)
    _floats(lse, (B, Hq, Lq), "lse")
    L = lib()
    ws, n = _workspace(workspace, L.gs_cross_attn_fwd_workspace_bytes(p), dev)
    _check(L.gs_cross_attn_fwd(p, _heads(q), _heads(k), _heads(v), _heads(out), _ptr(lse), _ptr(ws), n, _stream(stream)),
           "gs_cross_attn_fwd")
    return out, lse


def cross_attn_bwd(dout, q, k, v, out, lse, scale: float | None = None, ranges=None, key_mask=None, workspace=None,
                   stream=None) -> tuple:
    """gs_cross_attn_bwd: (dq, dk, dv) from the forward call's inputs and outputs and the gradient of out."""
    p = _attn_shape(q, k, v, scale, ranges, key_mask)
    dev = q.device
    _require(dout.shape == q.shape and out.shape == q.shape, "dout, out: q's shape")
    _type(q, dout, out)
    _floats(lse, (q.shape[0], q.shape[2], q.shape[1]), "lse")
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=dev) for x in (q, k, v))
    L = lib()
    ws, n = _workspace(workspace, L.gs_cross_attn_bwd_workspace_bytes(p), dev)
    _check(L.gs_cross_attn_bwd(p, _heads(dout), _heads(q), _heads(k), _heads(v), _heads(out), _ptr(lse), _heads(dq), _heads(dk),
                               _heads(dv), _ptr(ws), n, _stream(stream)), "gs_cross_attn_bwd")
    return dq, dk, dv


# -- gated activation with 8-bit checkpoints -------------------------------------------------


def _matrix(t, rows, width):
    _require(t.dim() == 2 and t.shape[0] == rows and t.shape[1] == width and (width <= 1 or t.stride(1) == 1),
             "matrices [rows][width] of one shape, rows dense")
    return t.data_ptr(), t.stride(0)


def gate8_fwd(gate, up, act: str = "silu", stream=None) -> tuple:
    """gs_gate8_fwd: (y, codes, bounds) of act(gate) * up; gate, up [rows, width] (views of one projection's output
    are taken as they are).  codes uint8 [2, rows, width] and bounds float32 [2, rows, blocks, 2] are what
    gate8_bwd needs."""
    _require(act in ACTS, f"act: one of {tuple(ACTS)}")
    _require(gate.dim() == 2, "matrices [rows][width]")
    rows, width = gate.shape
    dev, ty = gate.device, _type(gate, up)
    y = torch.empty((rows, width), dtype=gate.dtype, device=dev)
    codes = torch.empty((2, rows, width), dtype=torch.uint8, device=dev)
    bounds = torch.empty((2, rows, (width + CODE_BLOCK - 1) // CODE_BLOCK, 2), dtype=torch.float32, device=dev)
    _check(lib().gs_gate8_fwd(rows, width, ACTS[act], ty, *_matrix(gate, rows, width), *_matrix(up, rows, width),
                              *_matrix(y, rows, width), _ptr(codes), _ptr(bounds), _stream(stream)), "gs_gate8_fwd")
    return y, codes, bounds


def gate8_bwd(dy, codes, bounds, act: str = "silu", with_y: bool = True, dgate=None, dup=None, stream=None) -> tuple:
    """gs_gate8_bwd: (dgate, dup, y again or None) from the codes; ``dgate``, ``dup``: tensors to write to, such as the
    halves of one [rows, 2 * width] gradient."""
    _require(act in ACTS, f"act: one of {tuple(ACTS)}")
    _require(dy.dim() == 2, "matrices [rows][width]")
    rows, width = dy.shape
    dev = dy.device
    _require(codes.dtype == torch.uint8 and tuple(codes.shape) == (2, rows, width) and codes.is_contiguous()
             and codes.device == dev, "codes: gate8_fwd's")
    _floats(bounds, (2, rows, (width + CODE_BLOCK - 1) // CODE_BLOCK, 2), "bounds")
    dgate = torch.empty((rows, width), dtype=dy.dtype, device=dev) if dgate is None else dgate
    dup = torch.empty((rows, width), dtype=dy.dtype, device=dev) if dup is None else dup
    y = torch.empty((rows, width), dtype=dy.dtype, device=dev) if with_y else None
    ty = _type(dy, dgate, dup)
    _check(lib().gs_gate8_bwd(rows, width, ACTS[act], ty, *_matrix(dy, rows, width), _ptr(codes), _ptr(bounds),
                              *_matrix(dgate, rows, width), *_matrix(dup, rows, width),
                              *(_matrix(y, rows, width) if with_y else (None, 0)), _stream(stream)), "gs_gate8_bwd")
    return dgate, dup, y


# -- as differentiable torch functions -------------------------------------------------------


def _on_vectors(t):
    """t itself where the C calls take it as it is, a dense copy where they do not (an expanded gradient, say)."""
    each = 16 // t.element_size()
    dense = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s % each == 0 or n == 1 for s, n in zip(t.stride()[:-1], t.shape))
    return t if dense else t.contiguous()


class _NormRotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, pos_q, pos_k)
        ctx.more = (eps, pairs)
        return norm_rotate_fwd(q, k, wq, wk, cos, sin, pos_q, pos_k, eps, pairs)

    @staticmethod
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
        flat = h.reshape(-1, 2 * width)
        y, codes, bounds = gate8_fwd(flat[:, :width], flat[:, width:], act)
        ctx.save_for_backward(codes, bounds)
        ctx.act, ctx.shape = act, h.shape
        return y.view(*h.shape[:-1], width)

    @staticmethod
    def backward(ctx, dy):
        codes, bounds = ctx.saved_tensors
        width = codes.shape[2]
        dh = torch.empty((codes.shape[1], 2 * width), dtype=dy.dtype, device=dy.device)
        dy = dy.reshape(-1, width)
        dy = dy if dy.stride() == (width, 1) else dy.contiguous()
        gate8_bwd(dy, codes, bounds, ctx.act, False, dh[:, :width], dh[:, width:])
        return dh.view(ctx.shape), None


def gated8(h, act: str = "silu"):
    """act(gate) * up of a projection's output h [..., 2 * width] = (gate | up), with the gradient for h from 8-bit
    codes: between the passes only the codes and their bounds are kept, a quarter (float32) or half (bfloat16) of h."""
    return _Gated8.apply(h, act)
