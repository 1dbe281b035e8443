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
import functools
from typing import Optional

import numpy as np
import torch

import zero_sharded_mixed_reduce_amd as _z

ZSMR_FP32 = 3
TENSOR_CODES = {torch.float16: _z.ZSMR_FP16, torch.bfloat16: _z.ZSMR_BF16, torch.float32: ZSMR_FP32}
_NP64, _NP32 = np.dtype(np.int64), np.dtype(np.int32)
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
    """The entry points with every integer argument checked."""
    global _LIB
    if _LIB is None:
        _z.load()               # raises ImportError if the library has not been built
        _LIB = _z.checked_library(_z.LIB_PATH, SIGNATURES)
    return _LIB


def _raw(name: str):
    """An entry point whose integers come from tensors or are checked by its
    caller: the general check, 2 us a call, is left out."""
    fn = _RAW.get(name)
    if fn is None:
        fn = _RAW[name] = getattr(_lib(), name).fn
    return fn


_RAW: dict = {}
_CODE16 = {torch.float16: _z.ZSMR_FP16, torch.bfloat16: _z.ZSMR_BF16}


def _matrix(x, what: str, rows=None, width=None, dtype=None) -> tuple:
    """(rows, width, stride between rows, address) of a 16-bit matrix in device
    memory."""
    shape, t = x.shape, x.dtype
    if len(shape) != 2 or t not in _CODE16:
        raise ValueError(f"{what}: a matrix of 16-bit values is required, got {t} of {tuple(shape)}")
    if dtype is not None and t is not dtype:
        raise ValueError(f"{what}: {t}, the other operands are {dtype}")
    n, w = shape
    if width is not None and (n != rows or w != width):
        raise ValueError(f"{what}: {n} x {w}, {rows} x {width} is required")
    stride, one = x.stride()
    if one != 1 and w > 1:
        raise ValueError(f"{what}: elements of a row must be contiguous")
    if n <= 1:
        stride = w
    elif stride < w:
        raise ValueError(f"{what}: rows overlap")
    return n, w, stride, _ptr(x)


def _ids(ids) -> tuple:
    """(number, bytes of each, address) of a vector of token ids."""
    size, shape = _ID_BYTES.get(ids.dtype), ids.shape
    if size is None or len(shape) != 1 or not ids.is_contiguous():
        raise ValueError(f"token ids: a contiguous vector of int32 or int64 is required, got {ids.dtype} of {tuple(shape)}")
    return shape[0], size, _ptr(ids)


def _ptr(x) -> Optional[int]:
    """Device address of a tensor (a tensor in host memory is refused)."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"a {x.device.type} tensor was passed where device memory is required")
    return x.data_ptr()


def _vector(x, n: int, dtype, what: str) -> Optional[int]:
    """Address of a contiguous device vector of at least n elements (raw
    addresses are the caller's to check)."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype is not dtype or x.numel() < n or not x.is_contiguous():
        raise ValueError(f"{what}: at least {n} contiguous {dtype} are required, got {x.numel()} of {x.dtype}")
    return _ptr(x)


def _space(ws) -> tuple:
    """(address, bytes) of a workspace tensor."""
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("workspace: the tensor is not contiguous")
    return _ptr(ws), ws.numel() * ws.element_size()


def zsmr_embed_lookup(table, ids, out, scale: float = 1.0, stream=None) -> None:
    n, id_bytes, id_at = _ids(ids)
    vocab, width, ts, table_at = _matrix(table, "table")
    t = table.dtype
    _, _, os, out_at = _matrix(out, "out", n, width, t)
    code = _raw("zsmr_embed_lookup")(table_at, vocab, width, ts, _CODE16[t], id_at, id_bytes, n, scale,
                                     out_at, os, _z._stream(stream))
    if code:
        _z._check(code, "zsmr_embed_lookup")


def _size(n: int, where: str) -> int:
    if n < 0:
        raise _z.ZsmrError(_z.ZSMR_ERR_ARG, where)
    return n


def zsmr_embed_grad_workspace(vocab: int, width: int, n_tokens: int) -> int:
    return _size(_lib().zsmr_embed_grad_workspace(int(vocab), int(width), int(n_tokens)),
                 "zsmr_embed_grad_workspace")


def zsmr_embed_grad(dout, ids, dtable, ws, scale: float = 1.0, accumulate: bool = False,
                    stream=None) -> None:
    n, id_bytes, id_at = _ids(ids)
    vocab, width, ts, table_at = _matrix(dtable, "dtable")
    t = dtable.dtype
    _, _, ds, dout_at = _matrix(dout, "dout", n, width, t)
    code = _raw("zsmr_embed_grad")(dout_at, ds, _CODE16[t], id_at, id_bytes, n, vocab, width, scale,
                                   1 if accumulate else 0, table_at, ts, *_space(ws), _z._stream(stream))
    if code:
        _z._check(code, "zsmr_embed_grad")


def zsmr_xent_workspace(n_tokens: int, vocab: int, width: int, backward: bool = True) -> int:
    return _size(_lib().zsmr_xent_workspace(int(n_tokens), int(vocab), int(width),
                                            int(bool(backward))), "zsmr_xent_workspace")


def zsmr_xent_forward(x, w, labels, loss, lse, summary, ws, stream=None) -> None:
    """loss, lse: n_tokens fp32; summary: {mean loss, 1 / tokens that count,
    their number} fp32."""
    n, id_bytes, label_at = _ids(labels)
    vocab, width, wst, w_at = _matrix(w, "w")
    t = w.dtype
    _, _, xs, x_at = _matrix(x, "x", n, width, t)
    f = torch.float32
    code = _raw("zsmr_xent_forward")(x_at, xs, w_at, wst, _CODE16[t], label_at, id_bytes, n, vocab, width,
                                     _vector(loss, n, f, "loss"), _vector(lse, n, f, "lse"),
                                     _vector(summary, 3, f, "summary"), *_space(ws), _z._stream(stream))
    if code:
        _z._check(code, "zsmr_xent_forward")


def zsmr_xent_backward(x, w, labels, lse, dx, dw, ws, grad=None, scale=None,
                       accumulate: bool = False, stream=None) -> None:
    """dx or dw may be None; grad: n_tokens fp32 or None (ones); scale: one fp32
    on the device or None (1); accumulate adds to dw."""
    n, id_bytes, label_at = _ids(labels)
    vocab, width, wst, w_at = _matrix(w, "w")
    t = w.dtype
    _, _, xs, x_at = _matrix(x, "x", n, width, t)
    _, _, dxs, dx_at = _matrix(dx, "dx", n, width, t) if dx is not None else (0, 0, 0, None)
    _, _, dws, dw_at = _matrix(dw, "dw", vocab, width, t) if dw is not None else (0, 0, 0, None)
    f = torch.float32
    code = _raw("zsmr_xent_backward")(x_at, xs, w_at, wst, _CODE16[t], label_at, id_bytes, n, vocab, width,
                                      _vector(lse, n, f, "lse"), _vector(grad, n, f, "grad"),
                                      _vector(scale, 1, f, "scale"), dx_at, dxs, dw_at, dws,
                                      1 if accumulate else 0, *_space(ws), _z._stream(stream))
    if code:
        _z._check(code, "zsmr_xent_backward")


def _at(a) -> int:
    """Address of a numpy array (the quick way needs a writeable one)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except (TypeError, ValueError):
        return a.__array_interface__["data"][0]


def _list(tensors) -> tuple:
    """A tensor list's three arrays, and the arguments that stand for them."""
    if type(tensors) is tuple and len(tensors) == 3 and isinstance(tensors[0], np.ndarray):
        at, numels, dtypes = tensors
        n = len(at)
        for a, t in ((at, _NP64), (numels, _NP64), (dtypes, _NP32)):
            if a.dtype != t or a.shape != (n,) or not a.flags.c_contiguous:
                raise ValueError("tensor list: contiguous int64 addresses, int64 numels and int32 "
                                 "dtypes of one length are required")
    else:
        for i, x in enumerate(tensors):
            if not x.is_contiguous() or x.dtype not in TENSOR_CODES:
                raise ValueError(f"tensor list: tensor {i} is not contiguous fp16, bf16 or fp32")
        n = len(tensors)
        at = np.array([_ptr(x) for x in tensors], dtype=np.int64)
        numels = np.array([x.numel() for x in tensors], dtype=np.int64)
        dtypes = np.array([TENSOR_CODES[x.dtype] for x in tensors], dtype=np.int32)
    return (at, numels, dtypes), (_at(at), _at(numels), _at(dtypes), n)


def zsmr_norm_workspace(total: int, n_tensors: int) -> int:
    return _size(_lib().zsmr_norm_workspace(int(total), int(n_tensors)), "zsmr_norm_workspace")


def zsmr_grad_norm(tensors, max_norm: float, norm_coef, ws, eps: float = 1e-6, stream=None) -> None:
    """norm_coef: {norm, coefficient} fp32."""
    keep, args = _list(tensors)
    code = _raw("zsmr_grad_norm")(*args, max_norm, eps, _vector(norm_coef, 2, torch.float32, "norm_coef"),
                                  *_space(ws), _z._stream(stream))
    if code:
        _z._check(code, "zsmr_grad_norm")


def zsmr_clip_coef(sums, n: int, max_norm: float, norm_coef, eps: float = 1e-6, stream=None) -> None:
    _z._check(_lib().zsmr_clip_coef(_vector(sums, n, torch.float64, "sums"), n, max_norm, eps,
                                    _vector(norm_coef, 2, torch.float32, "norm_coef"),
                                    _z._stream(stream)), "zsmr_clip_coef")


def zsmr_clip_grads(tensors, coef, stream=None) -> None:
    keep, args = _list(tensors)
    code = _raw("zsmr_clip_grads")(*args, _vector(coef, 1, torch.float32, "coef"), _z._stream(stream))
    if code:
        _z._check(code, "zsmr_clip_grads")


def zsmr_clip_flatten(tensors, coef, flat, stream=None) -> None:
    keep, args = _list(tensors)
    t = flat.dtype
    if t not in _CODE16 or not flat.is_contiguous():
        raise ValueError(f"flat: a contiguous fp16 or bf16 tensor is required, got {t}")
    code = _raw("zsmr_clip_flatten")(*args, _vector(coef, 1, torch.float32, "coef"), _ptr(flat), flat.numel(),
                                     _CODE16[t], _z._stream(stream))
    if code:
        _z._check(code, "zsmr_clip_flatten")


def _piece(x, n: int, size: int, what: str) -> Optional[int]:
    """Address of n elements of `size` bytes (raw addresses are the caller's to
    check)."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_contiguous() or x.numel() * x.element_size() < n * size:
        _z._fits(x, n, size, what)
    return _ptr(x)


_I32, _I64 = 1 << 31, 1 << 63


def _checked_ints(name: str, i32, i64=()) -> None:
    for x in i32:
        if not -_I32 <= x < _I32:
            raise ValueError(f"{name}: {x} is outside int32")
    for x in i64:
        if not -_I64 <= x < _I64:
            raise ValueError(f"{name}: {x} is outside int64")


def zero_reduce_shard_sumsq(ctx, rank: int, unit: int, grads, row_stride: int, base_elem: int,
                            mean: bool, g_out, sumsq, ws, stream=None) -> None:
    _checked_ints("zero_reduce_shard_sumsq", (rank, unit), (row_stride, base_elem))
    n = _z._piece_len(ctx, rank, unit)
    _z._rows_fit(ctx, grads, row_stride, base_elem, n, "grads")
    code = _raw("zero_reduce_shard_sumsq")(ctx.handle, rank, unit, _ptr(grads), row_stride, base_elem,
                                           1 if mean else 0, _piece(g_out, n, 4, "g_out"),
                                           _vector(sumsq, 1, torch.float64, "sumsq"), *_space(ws),
                                           _z._stream(stream))
    if code:
        _z._check(code, "zero_reduce_shard_sumsq")


@functools.lru_cache(maxsize=16)
def _adam_ref(lr: float, beta1: float, beta2: float, eps: float):
    return ctypes.byref(_z._hp(lr, (beta1, beta2), eps))


def zero_clipped_step(ctx, rank: int, unit: int, g, coef, master, m, v, p16_dst, t: int, lr: float,
                      betas=(0.9, 0.999), eps: float = 1e-8, stream=None) -> None:
    _checked_ints("zero_clipped_step", (rank, unit, t))
    n = _z._piece_len(ctx, rank, unit)
    code = _raw("zero_clipped_step")(ctx.handle, rank, unit, _piece(g, n, 4, "g"),
                                     _vector(coef, 1, torch.float32, "coef"),
                                     _piece(master, n, 4, "master"), _piece(m, n, 4, "m"),
                                     _piece(v, n, 4, "v"), _piece(p16_dst, n, 2, "p16_dst"), t,
                                     _adam_ref(lr, *betas, eps), _z._stream(stream))
    if code:
        _z._check(code, "zero_clipped_step")
