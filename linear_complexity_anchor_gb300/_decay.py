"""Attention with decaying states: whole sequences, their gradients, and single tokens over a pool of states."""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from ._views import NO_VIEW, VIEW, Launch, empty_like, fail, library, rows_dtype, view

# anchor_attn_decay_t: dtype, B, heads, n, d, scale; Q, K, V, H, dH, dQ, dK, dV; log_decay, lengths, state, last, dlast, dstate
_pack = struct.Struct("=5if" + 8 * VIEW + "6Q").pack
# anchor_attn_decay_step_t: dtype, B, heads, n, d, slot_count, scale; Q, K, V, H; log_decay, states, slots
_pack_step = struct.Struct("=6if4x" + 4 * VIEW + "3Q").pack


def bind(lib) -> None:
    for name in ("anchor_attn_decay_forward", "anchor_attn_decay_backward", "anchor_attn_decay_step"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        fn.restype = ctypes.c_int


def _dense(t, name: str, dtype, shape, device: int) -> int:
    """The address of a dense tensor of this type and shape; 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be dense, {list(shape)}, on cuda:{device}")
    return t.data_ptr()


def _problem(Q, K, V, log_decay, scale):
    """The device, the structures' numbers, the views of Q, K and V, and the address of log_decay."""
    kind = rows_dtype(Q, "Q")
    dtype, device = Q.dtype, Q.get_device()
    views = (*view(Q, "Q", dtype, device), *view(K, "K", dtype, device), *view(V, "V", dtype, device))
    shape = Q.shape
    if K.shape != shape or V.shape != shape:
        raise ValueError("Q, K and V must be of one shape, [B, heads, n, d]")
    B, heads, n, d = shape
    if log_decay is None:
        raise TypeError("log_decay must be a float32 tensor [heads]")
    return device, (kind, B, heads, n, d), 1.0 / math.sqrt(d) if scale is None else scale, views, _dense(log_decay, "log_decay", torch.float32, (heads,), device)


def _call(fn: str, packed: bytes, handle: int) -> None:
    st = getattr(library(), fn)(packed, handle)
    if st:
        fail(st, fn)


def decay_forward(Q, K, V, log_decay, lengths=None, *, state=None, H=None, scale: float | None = None, return_state: bool = False,
                  stream=None):
    """H[i] = scale sum_{j <= i} exp((i - j) log_decay[head]) (q_i . k_j) v_j: linear attention whose state loses a part of
    itself with every token, in O(n).

    Q, K, V [B, heads, n, d] (bf16 or fp32; strides as they are, the last axis dense); log_decay: fp32 [heads], at most
    0; lengths: int32 [B] on the device, the tokens of each entry that count (None: all; the rows behind them are 0).
    state: fp32 [B, heads, d, d], the sum of k v^T (decayed) that the entries begin with; None: zeros.  scale defaults to
    1/sqrt(d).  Returns H in Q's order of axes, and with return_state the states behind the last tokens, which a next
    call or ``decay_step`` goes on from (in bf16 single bits of H may differ then).  A NaN or an infinity in K or V shows at the tokens from
    there on, and at those before it in its chunk: of the 128 (fp32: 64) from a multiple of that on.  Asynchronous on ``stream`` or the current stream."""
    device, numbers, scale, views, at_decay = _problem(Q, K, V, log_decay, scale)
    shape = Q.shape
    states = (shape[0], shape[1], shape[3], shape[3])
    at_lengths = _dense(lengths, "lengths", torch.int32, shape[:1], device)
    at_state = _dense(state, "state", torch.float32, states, device)
    at, last, given = Launch(device, stream), None, H
    with at as handle:
        if given is None:
            H, to = empty_like(Q)
        else:
            to = view(H, "H", Q.dtype, device)
            if H.shape != shape:
                raise ValueError("H must have Q's shape")
        if return_state:
            last = torch.empty(states, dtype=torch.float32, device=Q.device)
        _call("anchor_attn_decay_forward", _pack(*numbers, scale, *views, *to, *NO_VIEW, *NO_VIEW, *NO_VIEW, *NO_VIEW, at_decay, at_lengths,
                                                 at_state, last.data_ptr() if return_state else 0, 0, 0), handle)
    if at.stream is not None:
        at.used((Q, K, V, log_decay, lengths, state, given), (H if given is None else None, last))
    return (H, last) if return_state else H


def decay_backward(Q, K, V, dH, log_decay, lengths=None, *, state=None, dstate=None, scale: float | None = None, stream=None):
    """(dQ, dK, dV, dstate) for the upstream gradients dH of ``decay_forward``'s H and dstate (None: zero) of the states
    that it returns; the other arguments are those of that call.  The last is the gradient of its ``state``, None without
    one.  Rows from an entry's length on are zero.  A NaN or an infinity in Q or dH shows at dK and dV of the tokens up to
    there, and of those behind it in its chunk; in K or V as in the forward.  Heads or entries that share rows by an expanded axis get a gradient
    each; the decays get none."""
    device, numbers, scale, views, at_decay = _problem(Q, K, V, log_decay, scale)
    shape = Q.shape
    states = (shape[0], shape[1], shape[3], shape[3])
    g = view(dH, "dH", Q.dtype, device)
    if dH.shape != shape:
        raise ValueError("dH must have Q's shape")
    at_lengths = _dense(lengths, "lengths", torch.int32, shape[:1], device)
    at_state = _dense(state, "state", torch.float32, states, device)
    at_dlast = _dense(dstate, "dstate", torch.float32, states, device)
    at, first = Launch(device, stream), None
    with at as handle:
        (dQ, to_q), (dK, to_k), (dV, to_v) = empty_like(Q), empty_like(K), empty_like(V)
        if state is not None:
            first = torch.empty(states, dtype=torch.float32, device=Q.device)
        _call("anchor_attn_decay_backward", _pack(*numbers, scale, *views, *NO_VIEW, *g, *to_q, *to_k, *to_v, at_decay, at_lengths, at_state, 0,
                                                  at_dlast, 0 if first is None else first.data_ptr()), handle)
    if at.stream is not None:
        at.used((Q, K, V, dH, log_decay, lengths, state, dstate), (dQ, dK, dV, first))
    return dQ, dK, dV, first


def decay_step(Q, K, V, log_decay, states, slots=None, *, H=None, scale: float | None = None, stream=None):
    """``decay_forward`` for a few tokens (one, in serving) of B requests whose states are moved on in place.

    Q, K, V [B, heads, n, d]; states: fp32 [slots, heads, d, d]; slots: int32 [B] on the device, where each request's
    state lies (None: request b's is b).  A request whose slot is negative or past the last has H = 0 and moves no
    state; requests that share a slot are taken one after the other.  Returns H in Q's order of axes."""
    device, numbers, scale, views, at_decay = _problem(Q, K, V, log_decay, scale)
    shape = Q.shape
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise TypeError("states must be a float32 tensor [slots, heads, d, d]")
    at_states = _dense(states, "states", torch.float32, (states.shape[0], shape[1], shape[3], shape[3]), device)
    at_slots = _dense(slots, "slots", torch.int32, shape[:1], device)
    at, given = Launch(device, stream), H
    with at as handle:
        if given is None:
            H, to = empty_like(Q)
        else:
            to = view(H, "H", Q.dtype, device)
            if H.shape != shape:
                raise ValueError("H must have Q's shape")
        _call("anchor_attn_decay_step", _pack_step(*numbers, states.shape[0], scale, *views, *to, at_decay, at_states, at_slots), handle)
    if at.stream is not None:
        at.used((Q, K, V, log_decay, states, slots, given), (H if given is None else None,))
    return H
