"""Binding of the operators around the shard step (``include/zsmr_ops.h``).

Every function has the name of a C entry point.  Matrices are torch tensors
whose last dimension is contiguous (any stride between rows); their sizes,
strides and formats come from the tensors, which are checked against each
other before the library is called.  All arithmetic runs in its HIP kernels.

A list of gradient tensors is either a sequence of contiguous torch tensors, or
``(addresses, numels, dtypes)``: three numpy arrays (int64, int64, int32 format
codes) that a program may keep as long as its tensors stay where they are.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import numpy as np
import torch

import zero_sharded_mixed_reduce_amd as _z

ZSMR_FP32 = 3
TENSOR_CODES = {torch.float16: _z.ZSMR_FP16, torch.bfloat16: _z.ZSMR_BF16, torch.float32: ZSMR_FP32}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}

_i32, _i64, _vp, _f32, _f64 = (ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float,
                               ctypes.c_double)

# name -> (restype, argtypes); the list is the ABI of include/zsmr_ops.h
SIGNATURES = {
    "zsmr_embed_lookup": (_i32, [_vp, _i64, _i64, _i64, _i32, _vp, _i32, _i64, _f32, _vp, _i64, _vp]),
    "zsmr_embed_grad_workspace": (_i64, [_i64, _i64, _i64]),
    "zsmr_embed_grad": (_i32, [_vp, _i64, _i32, _vp, _i32, _i64, _i64, _i64, _f32, _i32, _vp, _i64,
                               _vp, _i64, _vp]),
    "zsmr_xent_workspace": (_i64, [_i64, _i64, _i64, _i32]),
    "zsmr_xent_forward": (_i32, [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp,
                                 _vp, _vp, _i64, _vp]),
    "zsmr_xent_backward": (_i32, [_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp,
                                  _vp, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp]),
    "zsmr_norm_workspace": (_i64, [_i64, _i32]),
    "zsmr_grad_norm": (_i32, [_vp, _vp, _vp, _i32, _f64, _f64, _vp, _vp, _i64, _vp]),
    "zsmr_clip_coef": (_i32, [_vp, _i64, _f64, _f64, _vp, _vp]),
    "zsmr_clip_grads": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp]),
    "zsmr_clip_flatten": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp, _i64, _i32, _vp]),
    "zero_reduce_shard_sumsq": (_i32, [_vp, _i32, _i32, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _i64,
                                       _vp]),
    "zero_clipped_step": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                 ctypes.POINTER(_z.zsmr_adam), _vp]),
}

_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        _z.load()               # raises ImportError if the library has not been built
        _LIB = _z.checked_library(_z.LIB_PATH, SIGNATURES)
    return _LIB


def _matrix(x, what: str, shape=None, dtype=None) -> tuple:
    """(rows, width, stride between rows) of a 16-bit matrix in device memory."""
    if x.dim() != 2 or x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"{what}: a matrix of 16-bit values is required, got {x.dtype} of {tuple(x.shape)}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{what}: {x.dtype}, the other operands are {dtype}")
    rows, width = x.shape
    if shape is not None and (rows, width) != tuple(shape):
        raise ValueError(f"{what}: {rows} x {width}, {shape[0]} x {shape[1]} is required")
    if width > 1 and x.stride(1) != 1:
        raise ValueError(f"{what}: elements of a row must be contiguous")
    stride = x.stride(0) if rows > 1 else width
    if stride < width:
        raise ValueError(f"{what}: rows overlap")
    return rows, width, stride


def _ids(ids, n: Optional[int] = None) -> int:
    """Bytes of one token id."""
    if ids.dim() != 1 or ids.dtype not in _ID_BYTES or not ids.is_contiguous():
        raise ValueError(f"token ids: a contiguous vector of int32 or int64 is required, got {ids.dtype} of {tuple(ids.shape)}")
    if n is not None and ids.numel() != n:
        raise ValueError(f"token ids: {ids.numel()}, {n} are required")
    return _ID_BYTES[ids.dtype]


def _vector(x, n: int, dtype, what: str) -> None:
    """A contiguous device vector of at least n elements (raw addresses are the
    caller's to check)."""
    if x is None or isinstance(x, int):
        return
    if x.dtype != dtype or not x.is_contiguous() or x.numel() < n:
        raise ValueError(f"{what}: at least {n} contiguous {dtype} are required, got {x.numel()} of {x.dtype}")


def _bytes(ws) -> int:
    """Bytes of a workspace tensor; a raw address carries no size."""
    if ws is None:
        return 0
    if not ws.is_contiguous():
        raise ValueError("workspace: the tensor is not contiguous")
    return ws.numel() * ws.element_size()


def zsmr_embed_lookup(table, ids, out, scale: float = 1.0, stream=None) -> None:
    vocab, width, ts = _matrix(table, "table")
    n, _, os = _matrix(out, "out", (ids.numel(), width), table.dtype)
    _z._check(_lib().zsmr_embed_lookup(_z._ptr(table), vocab, width, ts, TENSOR_CODES[table.dtype],
                                       _z._ptr(ids), _ids(ids), n, scale, _z._ptr(out), os,
                                       _z._stream(stream)), "zsmr_embed_lookup")


def _size(n: int, where: str) -> int:
    if n < 0:
        raise _z.ZsmrError(_z.ZSMR_ERR_ARG, where)
    return n


def zsmr_embed_grad_workspace(vocab: int, width: int, n_tokens: int) -> int:
    return _size(_lib().zsmr_embed_grad_workspace(int(vocab), int(width), int(n_tokens)),
                 "zsmr_embed_grad_workspace")


def zsmr_embed_grad(dout, ids, dtable, ws, scale: float = 1.0, accumulate: bool = False,
                    stream=None) -> None:
    vocab, width, ts = _matrix(dtable, "dtable")
    n, _, ds = _matrix(dout, "dout", (ids.numel(), width), dtable.dtype)
    _z._check(_lib().zsmr_embed_grad(_z._ptr(dout), ds, TENSOR_CODES[dtable.dtype], _z._ptr(ids),
                                     _ids(ids), n, vocab, width, scale, int(bool(accumulate)),
                                     _z._ptr(dtable), ts, _z._ptr(ws), _bytes(ws),
                                     _z._stream(stream)), "zsmr_embed_grad")


def zsmr_xent_workspace(n_tokens: int, vocab: int, width: int, backward: bool = True) -> int:
    return _size(_lib().zsmr_xent_workspace(int(n_tokens), int(vocab), int(width),
                                            int(bool(backward))), "zsmr_xent_workspace")


def zsmr_xent_forward(x, w, labels, loss, lse, summary, ws, stream=None) -> None:
    """loss, lse: n_tokens fp32; summary: {mean loss, 1 / tokens that count,
    their number} fp32."""
    vocab, width, wst = _matrix(w, "w")
    n, _, xs = _matrix(x, "x", (labels.numel(), width), w.dtype)
    _vector(loss, n, torch.float32, "loss")
    _vector(lse, n, torch.float32, "lse")
    _vector(summary, 3, torch.float32, "summary")
    _z._check(_lib().zsmr_xent_forward(_z._ptr(x), xs, _z._ptr(w), wst, TENSOR_CODES[w.dtype],
                                       _z._ptr(labels), _ids(labels), n, vocab, width, _z._ptr(loss),
                                       _z._ptr(lse), _z._ptr(summary), _z._ptr(ws), _bytes(ws),
                                       _z._stream(stream)), "zsmr_xent_forward")


def zsmr_xent_backward(x, w, labels, lse, dx, dw, ws, grad=None, scale=None,
                       accumulate: bool = False, stream=None) -> None:
    """dx or dw may be None; grad: n_tokens fp32 or None (ones); scale: one fp32
    on the device or None (1); accumulate adds to dw."""
    vocab, width, wst = _matrix(w, "w")
    n, _, xs = _matrix(x, "x", (labels.numel(), width), w.dtype)
    dxs = _matrix(dx, "dx", (n, width), w.dtype)[2] if dx is not None else 0
    dws = _matrix(dw, "dw", (vocab, width), w.dtype)[2] if dw is not None else 0
    _vector(lse, n, torch.float32, "lse")
    _vector(grad, n, torch.float32, "grad")
    _vector(scale, 1, torch.float32, "scale")
    _z._check(_lib().zsmr_xent_backward(_z._ptr(x), xs, _z._ptr(w), wst, TENSOR_CODES[w.dtype],
                                        _z._ptr(labels), _ids(labels), n, vocab, width, _z._ptr(lse),
                                        _z._ptr(grad), _z._ptr(scale), _z._ptr(dx), dxs, _z._ptr(dw),
                                        dws, int(bool(accumulate)), _z._ptr(ws), _bytes(ws),
                                        _z._stream(stream)), "zsmr_xent_backward")


def _list(tensors) -> tuple:
    """The three arrays of a tensor list."""
    if isinstance(tensors, tuple) and len(tensors) == 3 and isinstance(tensors[0], np.ndarray):
        at, numels, dtypes = tensors
        for a, t in ((at, np.int64), (numels, np.int64), (dtypes, np.int32)):
            if a.dtype != t or a.ndim != 1 or len(a) != len(at) or not a.flags.c_contiguous:
                raise ValueError("tensor list: contiguous int64 addresses, int64 numels and int32 "
                                 "dtypes of one length are required")
        return at, numels, dtypes
    for i, x in enumerate(tensors):
        if not x.is_contiguous() or x.dtype not in TENSOR_CODES:
            raise ValueError(f"tensor list: tensor {i} is not contiguous fp16, bf16 or fp32")
    return (np.array([_z._ptr(x) for x in tensors], dtype=np.int64),
            np.array([x.numel() for x in tensors], dtype=np.int64),
            np.array([TENSOR_CODES[x.dtype] for x in tensors], dtype=np.int32))


def zsmr_norm_workspace(total: int, n_tensors: int) -> int:
    return _size(_lib().zsmr_norm_workspace(int(total), int(n_tensors)), "zsmr_norm_workspace")


def zsmr_grad_norm(tensors, max_norm: float, norm_coef, ws, eps: float = 1e-6, stream=None) -> None:
    """norm_coef: {norm, coefficient} fp32."""
    at, numels, dtypes = _list(tensors)
    _vector(norm_coef, 2, torch.float32, "norm_coef")
    _z._check(_lib().zsmr_grad_norm(at.ctypes.data, numels.ctypes.data, dtypes.ctypes.data, len(at),
                                    max_norm, eps, _z._ptr(norm_coef), _z._ptr(ws), _bytes(ws),
                                    _z._stream(stream)), "zsmr_grad_norm")


def zsmr_clip_coef(sums, n: int, max_norm: float, norm_coef, eps: float = 1e-6, stream=None) -> None:
    _vector(sums, n, torch.float64, "sums")
    _vector(norm_coef, 2, torch.float32, "norm_coef")
    _z._check(_lib().zsmr_clip_coef(_z._ptr(sums), int(n), max_norm, eps, _z._ptr(norm_coef),
                                    _z._stream(stream)), "zsmr_clip_coef")


def zsmr_clip_grads(tensors, coef, stream=None) -> None:
    at, numels, dtypes = _list(tensors)
    _vector(coef, 1, torch.float32, "coef")
    _z._check(_lib().zsmr_clip_grads(at.ctypes.data, numels.ctypes.data, dtypes.ctypes.data, len(at),
                                     _z._ptr(coef), _z._stream(stream)), "zsmr_clip_grads")


def zsmr_clip_flatten(tensors, coef, flat, stream=None) -> None:
    at, numels, dtypes = _list(tensors)
    _vector(coef, 1, torch.float32, "coef")
    if flat.dtype not in (torch.float16, torch.bfloat16) or not flat.is_contiguous():
        raise ValueError(f"flat: a contiguous fp16 or bf16 tensor is required, got {flat.dtype}")
    _z._check(_lib().zsmr_clip_flatten(at.ctypes.data, numels.ctypes.data, dtypes.ctypes.data, len(at),
                                       _z._ptr(coef), _z._ptr(flat), flat.numel(),
                                       TENSOR_CODES[flat.dtype], _z._stream(stream)), "zsmr_clip_flatten")


def zero_reduce_shard_sumsq(ctx, rank: int, unit: int, grads, row_stride: int, base_elem: int,
                            mean: bool, g_out, sumsq, ws, stream=None) -> None:
    n = _z._piece_len(ctx, rank, unit)
    _z._rows_fit(ctx, grads, row_stride, base_elem, n, "grads")
    _z._fits(g_out, n, 4, "g_out")
    _vector(sumsq, 1, torch.float64, "sumsq")
    _z._check(_lib().zero_reduce_shard_sumsq(ctx.handle, rank, unit, _z._ptr(grads), int(row_stride),
                                             int(base_elem), int(bool(mean)), _z._ptr(g_out),
                                             _z._ptr(sumsq), _z._ptr(ws), _bytes(ws),
                                             _z._stream(stream)), "zero_reduce_shard_sumsq")


def zero_clipped_step(ctx, rank: int, unit: int, g, coef, master, m, v, p16_dst, t: int, lr: float,
                      betas=(0.9, 0.999), eps: float = 1e-8, stream=None) -> None:
    n = _z._piece_len(ctx, rank, unit)
    for x, what in ((g, "g"), (master, "master"), (m, "m"), (v, "v")):
        _z._fits(x, n, 4, what)
    _z._fits(p16_dst, n, 2, "p16_dst")
    _vector(coef, 1, torch.float32, "coef")
    hp = _z._hp(lr, betas, eps)
    _z._check(_lib().zero_clipped_step(ctx.handle, rank, unit, _z._ptr(g), _z._ptr(coef),
                                       _z._ptr(master), _z._ptr(m), _z._ptr(v), _z._ptr(p16_dst),
                                       int(t), ctypes.byref(hp), _z._stream(stream)),
              "zero_clipped_step")
