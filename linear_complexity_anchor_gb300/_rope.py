"""Rotary positions, and the norm of each head's query and key with the rotation in the same pass."""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

from ._views import NO_VIEW, Launch, View, check, empty_like, rows_dtype, view


class RopeTable(NamedTuple):
    """phases: int64 [axes, rot / 2], the part of a turn that one position adds to each pair's angle, as a 64-bit
    two's complement fraction; magnitude: the factor on the rotated columns."""
    phases: object
    magnitude: float = 1.0


class _Rope(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("d", ctypes.c_int), ("rot", ctypes.c_int), ("axes", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("norm", ctypes.c_int), ("weight_f32", ctypes.c_int),
                ("positions64", ctypes.c_int), ("eps", ctypes.c_float), ("magnitude", ctypes.c_float),
                ("phases", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    _fields_ = [("X", View), ("Y", View), ("dY", View), ("dX", View), ("weight", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("positions_batch", ctypes.c_longlong),
                ("start", ctypes.c_longlong), ("B", ctypes.c_int), ("heads", ctypes.c_int), ("n", ctypes.c_int)]


def bind(lib) -> None:
    for name in ("anchor_attn_norm_rope", "anchor_attn_norm_rope_backward"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(_Rope), ctypes.POINTER(_Rows), ctypes.POINTER(_Rows), ctypes.c_void_p]
        fn.restype = ctypes.c_int


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original: int | None = None, low: float = 1.0, high: float = 32.0, sections=None):
    """(radians that one position adds to each pair's angle as a list [axes][rot / 2], magnitude).

    theta_k = base^(-2 k / rot), k < rot / 2, and for long contexts, `factor` times as long as the one trained on:
      None      as it is
      "linear"  theta / factor
      "base"    base * factor^(rot / (rot - 2)) in the place of base: the slowest pair is stretched by factor, the
                fastest not at all (rot > 2)
      "bands"   a pair that makes more than `high` turns over `original` positions stays, one that makes fewer than
                `low` is divided by factor, between them theta g + theta / factor (1 - g) with
                g = (turns - low) / (high - low); magnitude 0.1 ln(factor) + 1
    sections: for several axes (the rows and columns of an image grid), the pairs that each axis turns; axis a's have
    base^(-k / sections[a]), k < sections[a], scaled alike."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and positive")
    if not (base > 0 and math.isfinite(base) and factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    parts = [rot // 2] if sections is None else [int(c) for c in sections]
    if not 1 <= len(parts) <= 3 or min(parts) < 1 or sum(parts) != rot // 2:
        raise ValueError("sections must be 1 to 3 positive numbers of pairs with the sum rot / 2")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "bands" and not (original is not None and original > 0 and high > low):
        raise ValueError("bands needs original > 0 and high > low")
    out, at = [], 0
    for pairs in parts:
        b = base
        if scaling == "base":
            if pairs < 2:
                raise ValueError('"base" needs two pairs at least for each axis')
            b = base * factor ** (pairs / (pairs - 1))
        row = [0.0] * (rot // 2)
        for k in range(pairs):
            theta = b ** (-k / pairs)
            if scaling == "linear":
                theta /= factor
            elif scaling == "bands":
                g = min(1.0, max(0.0, (original * theta / (2 * math.pi) - low) / (high - low)))
                theta = theta * g + theta / factor * (1 - g)
            row[at + k] = theta
        at += pairs
        out.append(row)
    return out, (0.1 * math.log(factor) + 1.0 if scaling == "bands" else 1.0)


def rope_table(rot: int, base: float = 10000.0, *, device="cuda", **how) -> RopeTable:
    """The table that ``rope`` and ``norm_rope`` take, for ``rope_frequencies(rot, base, **how)``; made once."""
    import torch
    theta, magnitude = rope_frequencies(rot, base, **how)
    turns = [[int(round(t / (2 * math.pi) * 2 ** 64)) % 2 ** 64 for t in row] for row in theta]
    signed = [[t - 2 ** 64 if t >= 2 ** 63 else t for t in row] for row in turns]
    return RopeTable(torch.tensor(signed, dtype=torch.int64).to(device), magnitude)


def _how(x, table, interleaved, norm, eps, weights, positions):
    import torch
    how = _Rope(dtype=rows_dtype(x, "the rows"), d=x.size(-1), axes=1, interleaved=1 if interleaved else 0, norm=norm, eps=eps,
                magnitude=1.0)
    if table is not None:
        phases, magnitude = table
        check(phases, "the table's phases", dim=2)
        if phases.dtype != torch.int64 or not phases.is_contiguous():
            raise TypeError("the table's phases must be contiguous int64")
        if phases.device != x.device:
            raise ValueError(f"the table must be on {x.device}")
        how.axes, how.rot, how.magnitude, how.phases = phases.size(0), 2 * phases.size(1), magnitude, phases.data_ptr()
    kinds = {p.dtype for p in positions if p is not None}
    if kinds:
        if len(kinds) > 1 or kinds - {torch.int32, torch.int64}:
            raise TypeError("positions must be int32 or int64, of one type")
        how.positions64 = 1 if torch.int64 in kinds else 0
    kinds = {w.dtype for w in weights if w is not None}
    if kinds:
        if len(kinds) > 1 or kinds - {x.dtype, torch.float32}:
            raise TypeError("weights must be of the rows' type or float32, and of one type")
        how.weight_f32 = 1 if torch.float32 in kinds else 0
    return how


def _rows(how, x, positions, start, weight, name):
    B, heads, n, d = x.shape
    if d != how.d:
        raise ValueError(f"{name} must have heads of {how.d}, got {d}")
    r = _Rows(X=NO_VIEW, Y=NO_VIEW, dY=NO_VIEW, dX=NO_VIEW, start=int(start), B=B, heads=heads, n=n)
    if positions is not None and how.rot:
        last = () if how.axes == 1 else (how.axes,)
        shape = tuple(positions.shape)
        if shape not in ((n, *last), (B, n, *last)):
            raise ValueError(f"positions of {name} must be {[n, *last]} or {[B, n, *last]}, got {list(shape)}")
        if not positions.is_cuda or positions.device != x.device:
            raise ValueError(f"positions must be on {x.device}")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        r.positions = positions.data_ptr()
        r.positions_batch = n * how.axes if len(shape) == 2 + len(last) else 0
    if weight is not None:
        check(weight, f"the weight of {name}", dim=1)
        if weight.size(0) != d or weight.device != x.device:
            raise ValueError(f"the weight of {name} must be [{d}] on {x.device}")
        r.weight = weight.data_ptr()
    return r


def _call(fn: str, how, first, second, handle) -> None:
    from . import _raise, load
    st = getattr(load(), fn)(ctypes.byref(how), ctypes.byref(first), ctypes.byref(second) if second is not None else None, handle)
    _raise(st, fn)


def _forward(X, table, positions, starts, weights, norm, eps, interleaved, out, stream):
    like = X[0]
    for x, name in zip(X, "QK"):
        if x is not None:
            check(x, name, like)
    how = _how(like, table, interleaved, norm, eps, weights, positions)
    rows = [None if x is None else _rows(how, x, p, s, w, name)
            for x, p, s, w, name in zip(X, positions, starts, weights, "QK")]
    at, Y = Launch(like.device, stream), []
    with at as handle:
        for x, r, y, name in zip(X, rows, out, "QK"):
            if x is not None:
                if y is None:
                    y = empty_like(x)
                else:
                    check(y, f"the output for {name}", x)
                    if y.shape != x.shape:
                        raise ValueError(f"the output for {name} must have its shape")
                r.X, r.Y = view(x), view(y)
            Y.append(y)
        _call("anchor_attn_norm_rope", how, rows[0], rows[1], handle)
    at.used((*X, *positions, *weights, table[0] if table is not None else None), Y)
    return Y


def rope(X, table, positions=None, *, start: int = 0, interleaved: bool = False, out=None, stream=None):
    """Turn the rows of X [B, heads, n, d] (bf16 or fp32; strides as they are, the last axis dense) by their
    positions: pairs (p, p + rot / 2) of the first rot columns, or (2p, 2p + 1) when interleaved; the other columns
    are passed through.

    table: from ``rope_table`` (or its (phases, magnitude)); positions: int32 or int64, [n] or [B, n], with the
    table's axes behind when there are several; None: start, start + 1, ...  out may be X itself.  Returns
    [B, heads, n, d] in X's order of axes.  Asynchronous on ``stream`` or the current stream."""
    if table is None:
        raise ValueError("rope needs a table")
    return _forward((X, None), table, (positions, None), (start, 0), (None, None), 0, 0.0, interleaved, (out, None), stream)[0]


def rope_backward(dY, table, positions=None, *, start: int = 0, interleaved: bool = False, stream=None):
    """dX for the upstream gradient dY of ``rope`` (turned back, by the same magnitude)."""
    if table is None:
        raise ValueError("rope_backward needs a table")
    check(dY, "dY")
    how = _how(dY, table, interleaved, 0, 0.0, (), (positions,))
    r = _rows(how, dY, positions, start, None, "dY")
    at = Launch(dY.device, stream)
    with at as handle:
        dX = empty_like(dY)
        r.dY, r.dX = view(dY), view(dX)
        _call("anchor_attn_norm_rope_backward", how, r, None, handle)
    at.used((dY, positions, table[0]), (dX,))
    return dX


def norm_rope(Q, K, table, *, q_weight=None, k_weight=None, q_positions=None, k_positions=None, q_start: int = 0,
              k_start: int = 0, eps: float = 1e-6, interleaved: bool = False, out=(None, None), stream=None):
    """(Q', K'): each row of Q [B, heads, n, d] and K [B', heads', n', d] divided by the root of its mean square
    (plus eps), times the weight [d] (of the rows' type or fp32; None: ones), then turned as ``rope`` turns it, in
    one launch.  K may be None (then K' is), and table None for the norms alone.  Anchors, which have no positions,
    go through a call of their own with table None.  The other arguments are ``rope``'s."""
    return tuple(_forward((Q, K), table, (q_positions, k_positions if K is not None else None), (q_start, k_start),
                          (q_weight, k_weight if K is not None else None), 1, eps, interleaved, out, stream))


def norm_rope_backward(Q, K, dQ, dK, table, *, q_weight=None, k_weight=None, q_positions=None, k_positions=None,
                       q_start: int = 0, k_start: int = 0, eps: float = 1e-6, interleaved: bool = False, stream=None):
    """(dQ, dK, dq_weight, dk_weight) for the upstream gradients dQ, dK of ``norm_rope``'s two results; Q and K are
    its inputs.  A weight's gradient is the sum over batch, heads and rows, in the weight's type; None without a weight.
    K = None leaves out its part."""
    X, G, W, P = (Q, K), (dQ, dK), (q_weight, k_weight), (q_positions, k_positions)
    if K is None:
        G, W, P = (dQ, None), (q_weight, None), (q_positions, None)
    for x, g, name in zip(X, G, "QK"):
        if x is not None:
            check(x, name, Q)
            check(g, f"d{name}", Q)
            if g.shape != x.shape:
                raise ValueError(f"d{name} must have {name}'s shape")
    how = _how(Q, table, interleaved, 1, eps, W, P)
    rows = [None if x is None else _rows(how, x, p, s, w, name) for x, p, s, w, name in zip(X, P, (q_start, k_start), W, "QK")]
    at, dX, dW = Launch(Q.device, stream), [], []
    with at as handle:
        import torch
        for x, g, w, r in zip(X, G, W, rows):
            dX.append(None if x is None else empty_like(x))
            dW.append(None if w is None else torch.empty_like(w))
            if x is not None:
                r.X, r.dY, r.dX = view(x), view(g), view(dX[-1])
                r.dweight = None if w is None else dW[-1].data_ptr()
        _call("anchor_attn_norm_rope_backward", how, rows[0], rows[1], handle)
    at.used((*X, *G, *W, *P, table[0] if table is not None else None), (*dX, *dW))
    return dX[0], dX[1], dW[0], dW[1]
