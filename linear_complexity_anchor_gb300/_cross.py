"""Cross attention to an encoder's states."""
from __future__ import annotations

import ctypes
import math

from ._views import Launch, View, check, empty_like, rows_dtype, view


class _Cross(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_int), ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("n", ctypes.c_int), ("s", ctypes.c_int), ("d", ctypes.c_int), ("scale", ctypes.c_float),
                ("Q", View), ("K", View), ("V", View), ("H", View), ("dH", View), ("dQ", View), ("dK", View),
                ("dV", View), ("lse", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


def bind(lib) -> None:
    for name in ("anchor_attn_cross_forward", "anchor_attn_cross_backward"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(_Cross), ctypes.c_void_p]
        fn.restype = ctypes.c_int


def _problem(Q, K, V, lengths, scale):
    import torch
    check(Q, "Q")
    check(K, "K", Q)
    check(V, "V", Q)
    B, heads, n, d = Q.shape
    if K.shape[0] != B or K.shape[3] != d or V.shape != K.shape:
        raise ValueError("Q is [B, heads, n, d]; K and V are [B, kv_heads, s, d]")
    p = _Cross(rows_dtype(Q, "Q"), B, heads, K.shape[1], n, K.shape[2], d, 1.0 / math.sqrt(d) if scale is None else scale,
               view(Q), view(K), view(V))
    if lengths is not None:
        if not isinstance(lengths, torch.Tensor) or lengths.dtype != torch.int32:
            raise TypeError("lengths must be an int32 tensor")
        if lengths.device != Q.device or tuple(lengths.shape) != (B,) or not lengths.is_contiguous():
            raise ValueError(f"lengths must be dense, [{B}], on {Q.device}")
        p.lengths = lengths.data_ptr()
    return p


def _call(fn: str, p, handle) -> None:
    from . import _raise, load
    _raise(getattr(load(), fn)(ctypes.byref(p), handle), fn)


def cross_forward(Q, K, V, lengths=None, *, H=None, scale: float | None = None, return_lse: bool = False, stream=None):
    """H[i] = sum_j softmax over j of (scale q_i . k_j) v_j over the first lengths[b] of an encoder's s states.

    Q [B, heads, n, d]; K, V [B, kv_heads, s, d] (bf16 or fp32; strides as they are, the last axis dense; heads a
    multiple of kv_heads: neighbouring query heads share a key head); lengths: int32 [B] on the device, None: all
    states.  An entry of length 0 has H = 0.  scale defaults to 1/sqrt(d).  Returns H [B, heads, n, d] in Q's order of
    axes, and with return_lse the logarithm of each row's sum, fp32 [B, heads, n], which ``cross_backward`` takes.
    Asynchronous on ``stream`` or the current stream."""
    import torch
    p = _problem(Q, K, V, lengths, scale)
    at, lse = Launch(Q.device, stream), None
    with at as handle:
        if H is None:
            H = empty_like(Q)
        else:
            check(H, "H", Q)
            if H.shape != Q.shape:
                raise ValueError("H must have Q's shape")
        p.H = view(H)
        if return_lse:
            lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
            p.lse = lse.data_ptr()
        _call("anchor_attn_cross_forward", p, handle)
    at.used((Q, K, V, lengths), (H, lse))
    return (H, lse) if return_lse else H


def cross_backward(Q, K, V, H, lse, dH, lengths=None, *, scale: float | None = None, stream=None):
    """(dQ, dK, dV) for the upstream gradient dH of ``cross_forward``'s H; H and lse are its results for the same
    Q, K, V, lengths and scale.  Rows of dK and dV from an entry's length on are zero.  K or V that entries share by
    an expanded axis get a gradient for each entry."""
    import torch
    p = _problem(Q, K, V, lengths, scale)
    for t, name in ((H, "H"), (dH, "dH")):
        check(t, name, Q)
        if t.shape != Q.shape:
            raise ValueError(f"{name} must have Q's shape")
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or lse.device != Q.device:
        raise TypeError(f"lse must be a float32 tensor on {Q.device}")
    if lse.shape != Q.shape[:3] or not lse.is_contiguous():
        raise ValueError("lse must be dense, [B, heads, n]")
    at = Launch(Q.device, stream)
    with at as handle:
        dQ, dK, dV = empty_like(Q), empty_like(K), empty_like(V)
        p.H, p.dH, p.dQ, p.dK, p.dV, p.lse = view(H), view(dH), view(dQ), view(dK), view(dV), lse.data_ptr()
        _call("anchor_attn_cross_backward", p, handle)
    at.used((Q, K, V, H, lse, dH, lengths), (dQ, dK, dV))
    return dQ, dK, dV
