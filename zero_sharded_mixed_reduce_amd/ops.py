"""Binding of the operators around the shard step (``include/zsmr_ops.h``).

Every function has the name of a C entry point; the checks and the calls are in
the extension module ``_ops`` (``csrc/zsmr_python.cpp``).  Matrices are torch tensors
whose last dimension is contiguous (any stride between rows); their sizes,
strides and formats come from the tensors, which are checked against each
other before the library is called.  Vectors of floats and workspaces may also be raw device
addresses, whose lengths are the caller's to check.  All arithmetic runs in the
library's HIP kernels.

A list of gradient tensors is either any iterable of contiguous torch tensors, or
``(addresses, numels, dtypes)``: three numpy arrays (int64, int64, int32 format
codes) that a program may keep as long as its tensors stay where they are.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

import zero_sharded_mixed_reduce_amd as _z

_z.load()                       # raises ImportError if the libraries have not been built
from . import _ops  # noqa: E402  (the native half: checks of tensors, calls of libzsmr.so)

ZSMR_FP32 = 3
TENSOR_CODES = {torch.float16: _z.ZSMR_FP16, torch.bfloat16: _z.ZSMR_BF16, torch.float32: ZSMR_FP32}

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
        _LIB = _z.checked_library(_z.LIB_PATH, SIGNATURES)
    return _LIB


def _size(n: int, where: str) -> int:
    if n < 0:
        raise _z.ZsmrError(_z.ZSMR_ERR_ARG, where)
    return n


def zsmr_embed_lookup(table, ids, out, scale: float = 1.0, stream=None) -> None:
    code = _ops.embed_lookup(table, ids, out, scale, stream)
    if code:
        _z._check(code, "zsmr_embed_lookup")


def zsmr_embed_grad_workspace(vocab: int, width: int, n_tokens: int) -> int:
    return _size(_lib().zsmr_embed_grad_workspace(int(vocab), int(width), int(n_tokens)),
                 "zsmr_embed_grad_workspace")


def zsmr_embed_grad(dout, ids, dtable, ws, scale: float = 1.0, accumulate: bool = False,
                    stream=None) -> None:
    code = _ops.embed_grad(dout, ids, dtable, ws, scale, accumulate, stream)
    if code:
        _z._check(code, "zsmr_embed_grad")


def zsmr_xent_workspace(n_tokens: int, vocab: int, width: int, backward: bool = True) -> int:
    return _size(_lib().zsmr_xent_workspace(int(n_tokens), int(vocab), int(width),
                                            int(bool(backward))), "zsmr_xent_workspace")


def zsmr_xent_forward(x, w, labels, loss, lse, summary, ws, stream=None) -> None:
    """loss, lse: n_tokens fp32; summary: {mean loss, 1 / tokens that count,
    their number} fp32."""
    code = _ops.xent_forward(x, w, labels, loss, lse, summary, ws, stream)
    if code:
        _z._check(code, "zsmr_xent_forward")


def zsmr_xent_backward(x, w, labels, lse, dx, dw, ws, grad=None, scale=None,
                       accumulate: bool = False, stream=None) -> None:
    """dx or dw may be None; grad: n_tokens fp32 or None (ones); scale: one fp32
    on the device or None (1); accumulate adds to dw."""
    code = _ops.xent_backward(x, w, labels, lse, dx, dw, ws, grad, scale, accumulate, stream)
    if code:
        _z._check(code, "zsmr_xent_backward")


def _list(tensors) -> tuple:
    """A tensor list's three arrays."""
    if type(tensors) is tuple and len(tensors) == 3 and isinstance(tensors[0], np.ndarray):
        return tensors
    tensors = list(tensors)         # gone through more than once below
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
    code = _ops.grad_norm(at, numels, dtypes, max_norm, norm_coef, ws, eps, stream)
    if code:
        _z._check(code, "zsmr_grad_norm")


def zsmr_clip_coef(sums, n: int, max_norm: float, norm_coef, eps: float = 1e-6, stream=None) -> None:
    code = _ops.clip_coef(sums, n, max_norm, norm_coef, eps, stream)
    if code:
        _z._check(code, "zsmr_clip_coef")


def zsmr_clip_grads(tensors, coef, stream=None) -> None:
    at, numels, dtypes = _list(tensors)
    code = _ops.clip_grads(at, numels, dtypes, coef, stream)
    if code:
        _z._check(code, "zsmr_clip_grads")


def zsmr_clip_flatten(tensors, coef, flat, stream=None) -> None:
    at, numels, dtypes = _list(tensors)
    code = _ops.clip_flatten(at, numels, dtypes, coef, flat, stream)
    if code:
        _z._check(code, "zsmr_clip_flatten")


def zero_reduce_shard_sumsq(ctx, rank: int, unit: int, grads, row_stride: int, base_elem: int,
                            mean: bool, g_out, sumsq, ws, stream=None) -> None:
    code = _ops.reduce_shard_sumsq(ctx.handle, rank, unit, grads, row_stride, base_elem, mean, g_out,
                                   sumsq, ws, stream)
    if code:
        _z._check(code, "zero_reduce_shard_sumsq")


def zero_clipped_step(ctx, rank: int, unit: int, g, coef, master, m, v, p16_dst, t: int, lr: float,
                      betas=(0.9, 0.999), eps: float = 1e-8, stream=None) -> None:
    beta1, beta2 = betas
    code = _ops.clipped_step(ctx.handle, rank, unit, g, coef, master, m, v, p16_dst, t, lr, beta1,
                             beta2, eps, stream)
    if code:
        _z._check(code, "zero_clipped_step")
