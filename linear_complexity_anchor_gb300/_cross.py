"""Cross attention to an encoder's states."""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from ._views import NO_VIEW, VIEW, Launch, empty_like, fail, library, rows_dtype, view

# anchor_attn_cross_t: dtype, B, heads, kv_heads, n, s, d, scale; Q, K, V, H, dH, dQ, dK, dV; lse, lengths
_pack = struct.Struct("=7if" + 8 * VIEW + "QQ").pack


def bind(lib) -> None:
    for name in ("anchor_attn_cross_forward", "anchor_attn_cross_backward"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        fn.restype = ctypes.c_int


def _problem(Q, K, V, lengths, scale):
    """The device, the structure's numbers, its views of Q, K and V, and the lengths' pointer."""
    kind = rows_dtype(Q, "Q")
    dtype, device = Q.dtype, Q.get_device()
    views = (*view(Q, "Q", dtype, device), *view(K, "K", dtype, device), *view(V, "V", dtype, device))
    B, heads, n, d = Q.shape
    Bk, kv, s, dk = shape = K.shape
    if Bk != B or dk != d or V.shape != shape:
        raise ValueError("Q is [B, heads, n, d]; K and V are [B, kv_heads, s, d]")
    at = 0
    if lengths is not None:
        if not isinstance(lengths, torch.Tensor) or lengths.dtype is not torch.int32:
            raise TypeError("lengths must be an int32 tensor")
        if lengths.get_device() != device or lengths.shape != (B,) or not lengths.is_contiguous():
            raise ValueError(f"lengths must be dense, [{B}], on cuda:{device}")
        at = lengths.data_ptr()
    return device, (kind, B, heads, kv, n, s, d, 1.0 / math.sqrt(d) if scale is None else scale), views, at


def _call(fn: str, packed: bytes, handle: int) -> None:
    st = getattr(library(), fn)(packed, handle)
    if st:
        fail(st, fn)


def cross_forward(Q, K, V, lengths=None, *, H=None, scale: float | None = None, return_lse: bool = False, stream=None):
    """H[i] = sum_j softmax over j of (scale q_i . k_j) v_j over the first lengths[b] of an encoder's s states.

    Q [B, heads, n, d]; K, V [B, kv_heads, s, d] (bf16 or fp32; strides as they are, the last axis dense; heads a
    multiple of kv_heads: neighbouring query heads share a key head); lengths: int32 [B] on the device, None: all
    states.  An entry of length 0 has H = 0.  scale defaults to 1/sqrt(d).  Returns H [B, heads, n, d] in Q's order of
    axes, and with return_lse the logarithm of each row's sum, fp32 [B, heads, n], which ``cross_backward`` takes.
    Asynchronous on ``stream`` or the current stream."""
    device, numbers, views, at_lengths = _problem(Q, K, V, lengths, scale)
    at, lse, given = Launch(device, stream), None, H
    with at as handle:
        if given is None:
            H, to = empty_like(Q)
        else:
            to = view(H, "H", Q.dtype, device)
            if H.shape != Q.shape:
                raise ValueError("H must have Q's shape")
        if return_lse:
            lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
        _call("anchor_attn_cross_forward", _pack(*numbers, *views, *to, *NO_VIEW, *NO_VIEW, *NO_VIEW, *NO_VIEW,
                                                 lse.data_ptr() if return_lse else 0, at_lengths), handle)
    if at.stream is not None:
        at.used((Q, K, V, lengths, given), (H if given is None else None, lse))
    return (H, lse) if return_lse else H


def cross_backward(Q, K, V, H, lse, dH, lengths=None, *, scale: float | None = None, stream=None):
    """(dQ, dK, dV) for the upstream gradient dH of ``cross_forward``'s H; H and lse are its results for the same
    Q, K, V, lengths and scale.  Rows of dK and dV from an entry's length on are zero.  K or V that entries share by
    an expanded axis get a gradient for each entry."""
    device, numbers, views, at_lengths = _problem(Q, K, V, lengths, scale)
    dtype, shape = Q.dtype, Q.shape
    views += (*view(H, "H", dtype, device), *view(dH, "dH", dtype, device))
    if H.shape != shape or dH.shape != shape:
        raise ValueError("H and dH must have Q's shape")
    if not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32 or lse.get_device() != device:
        raise TypeError(f"lse must be a float32 tensor on cuda:{device}")
    if lse.shape != shape[:3] or not lse.is_contiguous():
        raise ValueError("lse must be dense, [B, heads, n]")
    at = Launch(device, stream)
    with at as handle:
        (dQ, to_q), (dK, to_k), (dV, to_v) = empty_like(Q), empty_like(K), empty_like(V)
        _call("anchor_attn_cross_backward", _pack(*numbers, *views, *to_q, *to_k, *to_v, lse.data_ptr(), at_lengths), handle)
    if at.stream is not None:
        at.used((Q, K, V, H, lse, dH, lengths), (dQ, dK, dV))
    return dQ, dK, dV
