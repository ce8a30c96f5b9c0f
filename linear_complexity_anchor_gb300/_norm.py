"""The RMS norm of a residual sum, with a result in 16, 32 or 8 bits, and its backward."""
from __future__ import annotations

import ctypes
import struct

import torch

from ._views import NO_VIEW, VIEW, Launch, fail, library, rows_dtype

# anchor_attn_add_norm_t: dtype, B, n, D, weight_f32, bits8, group, eps; X, R, S, Y, dY, dS, dX; weight, dweight, scales
_pack = struct.Struct("=7if" + 7 * VIEW + "QQQ").pack
GROUPS = (0, 32, 64, 128)


def bind(lib) -> None:
    for name in ("anchor_attn_add_norm", "anchor_attn_add_norm_backward"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        fn.restype = ctypes.c_int


def _rows(t, name: str, like=None) -> tuple:
    """The packed view of a [n, D] or [B, n, D] tensor whose last axis is dense; of `like`'s shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if like is not None:
        if t.dtype is not like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.get_device() != like.get_device():
            raise ValueError(f"{name} must be on {like.device}, got {t.device}")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have the shape {tuple(like.shape)}, got {tuple(t.shape)}")
    strides = t.stride()
    if len(strides) not in (2, 3):
        raise ValueError(f"{name} must be [n, D] or [B, n, D]")
    if strides[-1] != 1 and t.size(-1) > 1:
        raise ValueError(f"the last axis of {name} must be dense")
    return t.data_ptr(), strides[0] if len(strides) == 3 else 0, 0, strides[-2]


def _numbers(x, weight, eps, bits8=0, group=0) -> tuple:
    kind, shape = rows_dtype(x, "the rows"), x.shape
    wide = 0
    if weight is not None:
        if not isinstance(weight, torch.Tensor):
            raise TypeError("weight must be a torch.Tensor")
        wide = 1 if weight.dtype is torch.float32 else 0
        if not wide and weight.dtype is not x.dtype:
            raise TypeError("weight must be of the rows' type or float32")
        if weight.shape != shape[-1:] or weight.get_device() != x.get_device() or not weight.is_contiguous():
            raise ValueError(f"weight must be dense, [{shape[-1]}], on {x.device}")
    return kind, shape[0] if len(shape) == 3 else 1, shape[-2], shape[-1], wide, bits8, group, eps


def _call(fn: str, packed: bytes, handle: int) -> None:
    st = getattr(library(), fn)(packed, handle)
    if st:
        fail(st, fn)


def _dense(x, dtype):
    """An empty tensor of x's shape, and its view."""
    y = torch.empty(x.shape, dtype=dtype, device=x.device)
    strides = y.stride()
    return y, (y.data_ptr(), strides[0] if len(strides) == 3 else 0, 0, strides[-2])


def _forward(X, R, weight, eps, S, bits8, group, stream):
    if R is None and S is not None:
        raise ValueError("S is written where R is given")
    x = _rows(X, "X")
    numbers = _numbers(X, weight, eps, bits8, group)
    r = NO_VIEW if R is None else _rows(R, "R", X)
    at, given, scales = Launch(X.get_device(), stream), S, None
    with at as handle:
        s = NO_VIEW
        if R is None:
            S = X
        elif S is None:
            S, s = _dense(X, X.dtype)
        else:
            s = _rows(S, "S", X)
        Y, y = _dense(X, torch.float8_e4m3fn if bits8 else X.dtype)
        if bits8:
            groups = -(-X.shape[-1] // group) if group else 1
            scales = torch.empty((*X.shape[:-1], groups), dtype=torch.float32, device=X.device)
        _call("anchor_attn_add_norm", _pack(*numbers, *x, *r, *s, *y, *NO_VIEW, *NO_VIEW, *NO_VIEW,
                                            0 if weight is None else weight.data_ptr(), 0, 0 if scales is None else scales.data_ptr()), handle)
    if at.stream is not None:
        at.used((X, R, weight, given), (Y, scales, S if R is not None and given is None else None))
    return Y, scales, S


def add_norm(X, R=None, weight=None, *, eps: float = 1e-6, S=None, stream=None):
    """(Y, S): the residual sum S = X + R in the rows' type, and its norm Y = weight S / sqrt(mean(S^2) + eps).

    X, R: [n, D] or [B, n, D] (bf16 or fp32; strides as they are, the last axis dense; D a multiple of 16 up to
    16384); weight: [D], of the rows' type or fp32 (None: ones).  Rows may be of any finite size; those of zeros have Y = 0, with
    eps = 0 too.  Without R the norm is X's, and S is X.  S may be
    given, to write the sum over X or R or elsewhere.  Asynchronous on ``stream`` or the current stream."""
    Y, _, S = _forward(X, R, weight, eps, S, 0, 0, stream)
    return Y, S


def add_norm_8bit(X, R=None, weight=None, *, eps: float = 1e-6, group: int = 0, S=None, stream=None):
    """(Y, scales, S): as ``add_norm``, with Y in 8 bits (float8_e4m3fn) for the product behind it.

    Y scales stands for the norm: scales are fp32 [n, groups] (or [B, n, groups]), one for each row, or with group =
    32, 64 or 128 for each so many columns: the largest magnitude among them over 448.  Columns of zeros have scale 0."""
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}")
    return _forward(X, R, weight, eps, S, 1, group, stream)


def add_norm_backward(S, dY, weight=None, *, dS=None, eps: float = 1e-6, stream=None):
    """(dX, dweight) for the upstream gradients dY of ``add_norm``'s Y and dS (or None) of its S, which is given.  dX is
    the gradient of X and of R alike; dweight is summed over the rows, in the weight's type; None without a weight."""
    s = _rows(S, "S")
    numbers = _numbers(S, weight, eps)
    dy, ds = _rows(dY, "dY", S), NO_VIEW if dS is None else _rows(dS, "dS", S)
    at = Launch(S.get_device(), stream)
    with at as handle:
        dX, dx = _dense(S, S.dtype)
        dweight = None if weight is None else torch.empty_like(weight)
        _call("anchor_attn_add_norm_backward", _pack(*numbers, *NO_VIEW, *NO_VIEW, *s, *NO_VIEW, *dy, *ds, *dx, 0 if weight is None else weight.data_ptr(),
                                                     0 if dweight is None else dweight.data_ptr(), 0), handle)
    if at.stream is not None:
        at.used((S, dY, weight, dS), (dX, dweight))
    return dX, dweight
