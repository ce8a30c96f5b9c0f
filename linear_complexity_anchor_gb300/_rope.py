"""Rotary positions, and the norm of each head's query and key with the rotation in the same pass."""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from ._views import NO_VIEW, VIEW, Launch, empty_like, fail, library, rows_dtype, view


class RopeTable(NamedTuple):
    """phases: int64 [axes, rot / 2], the part of a turn that one position adds to each pair's angle, as a 64-bit
    two's complement fraction; magnitude: the factor on the rotated columns."""
    phases: object
    magnitude: float = 1.0


# anchor_attn_rope_t: dtype, d, rot, axes, interleaved, norm, weight_f32, positions64; eps, magnitude; phases
_pack_how = struct.Struct("=8i2fQ").pack
# anchor_attn_rows_t: X, Y, dY, dX; weight, dweight, positions; positions_batch, start; B, heads, n
_pack_rows = struct.Struct("=" + 4 * VIEW + "QQQqq3i4x").pack


def bind(lib) -> None:
    for name in ("anchor_attn_norm_rope", "anchor_attn_norm_rope_backward"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.c_void_p] * 4
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
    theta, magnitude = rope_frequencies(rot, base, **how)
    turns = [[int(round(t / (2 * math.pi) * 2 ** 64)) % 2 ** 64 for t in row] for row in theta]
    signed = [[t - 2 ** 64 if t >= 2 ** 63 else t for t in row] for row in turns]
    return RopeTable(torch.tensor(signed, dtype=torch.int64).to(device), magnitude)


def _how(x, table, interleaved, norm, eps, weights, positions):
    """The packed anchor_attn_rope_t, and (d, rot, axes, device)."""
    kind, dtype, device = rows_dtype(x, "the rows"), x.dtype, x.get_device()
    axes, rot, magnitude, at = 1, 0, 1.0, 0
    if table is not None:
        phases, magnitude = table
        if not isinstance(phases, torch.Tensor) or phases.dtype is not torch.int64 or phases.dim() != 2 or not phases.is_contiguous():
            raise TypeError("the table's phases must be a contiguous int64 tensor [axes, rot / 2]")
        if phases.get_device() != device:
            raise ValueError(f"the table must be on cuda:{device}")
        axes, rot = phases.shape
        rot, at = 2 * rot, phases.data_ptr()
    wide = long = -1  # not yet known
    for p in positions:
        if p is not None:
            here = 1 if p.dtype is torch.int64 else 0
            if (not here and p.dtype is not torch.int32) or long == 1 - here:
                raise TypeError("positions must be int32 or int64, of one type")
            long = here
    for w in weights:
        if w is not None:
            here = 1 if w.dtype is torch.float32 else 0
            if (not here and w.dtype is not dtype) or wide == 1 - here:
                raise TypeError("weights must be of the rows' type or float32, and of one type")
            wide = here
    d = x.shape[-1]
    return _pack_how(kind, d, rot, axes, 1 if interleaved else 0, norm, max(wide, 0), max(long, 0), eps, magnitude, at), (d, rot, axes, device)


def _rows(size, X, Y, dY, dX, shape, positions, start, weight, dweight, name):
    """The packed anchor_attn_rows_t of one tensor of this shape; X ... dX are its views."""
    d, rot, axes, device = size
    B, heads, n, width = shape
    if width != d:
        raise ValueError(f"{name} must have heads of {d}, got {width}")
    at = batch = 0
    if positions is not None and rot:
        last = () if axes == 1 else (axes,)
        of = positions.shape
        if of == (B, n, *last):
            batch = n * axes
        elif of != (n, *last):
            raise ValueError(f"positions of {name} must be {[n, *last]} or {[B, n, *last]}, got {list(of)}")
        if positions.get_device() != device:
            raise ValueError(f"positions must be on cuda:{device}")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        at = positions.data_ptr()
    if weight is not None and (weight.shape != (d,) or weight.get_device() != device or not weight.is_contiguous()):
        raise ValueError(f"the weight of {name} must be dense, [{d}], on cuda:{device}")
    return _pack_rows(*X, *Y, *dY, *dX, 0 if weight is None else weight.data_ptr(), 0 if dweight is None else dweight.data_ptr(),
                      at, batch, start, B, heads, n)


def _call(fn: str, how: bytes, first: bytes, second, handle: int) -> None:
    st = getattr(library(), fn)(how, first, second, handle)
    if st:
        fail(st, fn)


def _forward(X, table, positions, starts, weights, norm, eps, interleaved, out, stream):
    how, size = _how(X[0], table, interleaved, norm, eps, weights, positions)
    dtype, device = X[0].dtype, size[3]
    views = [None if x is None else view(x, name, dtype, device) for x, name in zip(X, "QK")]
    at, Y, rows = Launch(device, stream), [None, None], [None, None]
    with at as handle:
        for i, x in enumerate(X):
            if x is None:
                continue
            name, y, shape = "QK"[i], out[i], x.shape
            if y is None:
                y, to = empty_like(x)
            else:
                to = view(y, f"the output for {name}", dtype, device)
                if y.shape != shape:
                    raise ValueError(f"the output for {name} must have its shape")
            Y[i] = y
            rows[i] = _rows(size, views[i], to, NO_VIEW, NO_VIEW, shape, positions[i], starts[i], weights[i], None, name)
        _call("anchor_attn_norm_rope", how, rows[0], rows[1], handle)
    if at.stream is not None:
        at.used((*X, *positions, *weights, table[0] if table is not None else None, *out), [y for y, o in zip(Y, out) if o is None])
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
    how, size = _how(dY, table, interleaved, 0, 0.0, (), (positions,))
    g = view(dY, "dY", dY.dtype, size[3])
    at = Launch(size[3], stream)
    with at as handle:
        dX, to = empty_like(dY)
        rows = _rows(size, NO_VIEW, NO_VIEW, g, to, dY.shape, positions, start, None, None, "dY")
        _call("anchor_attn_norm_rope_backward", how, rows, None, handle)
    if at.stream is not None:
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
    how, size = _how(Q, table, interleaved, 1, eps, W, P)
    dtype, device = Q.dtype, size[3]
    views = [None if x is None else (view(x, name, dtype, device), view(g, f"d{name}", dtype, device)) for x, g, name in zip(X, G, "QK")]
    at, dX, dW, rows = Launch(device, stream), [None, None], [None, None], [None, None]
    with at as handle:
        for i, x in enumerate(X):
            if x is None:
                continue
            name, shape, w = "QK"[i], x.shape, W[i]
            dX[i], to = empty_like(x)
            if w is not None:
                dW[i] = torch.empty_like(w)
            if G[i].shape != shape:
                raise ValueError(f"d{name} must have {name}'s shape")
            rows[i] = _rows(size, views[i][0], NO_VIEW, views[i][1], to, shape, P[i], (q_start, k_start)[i], w, dW[i], name)
        _call("anchor_attn_norm_rope_backward", how, rows[0], rows[1], handle)
    if at.stream is not None:
        at.used((*X, *G, *W, *P, table[0] if table is not None else None), (*dX, *dW))
    return dX[0], dX[1], dW[0], dW[1]
