"""64-bit references of cross attention, rotary positions and normalised rotary rows, each with a bound on what the
roundings of the kernels can add up to, element by element.

Roundings: u is half a step of the rows' type (a result rounded to it is off by u |result| at most), f half a step of
fp32.  A sum of k products in fp32 is off by (k + 1) f times the sum of the products' magnitudes at most, in any order.
Exponentials, sines and reciprocals are off by a few f; E = 16 f stands for all that one element meets of them."""
import math

import torch

F = 2.0 ** -24
E = 16 * F


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def cross_reference(Q, K, V, lengths, scale, dH=None):
    """{name: (value, bound)} for H, lse and, with dH, dQ, dK, dV (all [B, heads, ...] in 64 bits on Q's device)."""
    u = half_step(Q.dtype)
    up = u if Q.dtype == torch.bfloat16 else 0.0  # the weights P and dS meet the second product in the rows' type
    B, heads, n, d = Q.shape
    kv, s = K.shape[1], K.shape[2]
    group = heads // kv
    L = torch.full((B,), s, dtype=torch.int64) if lengths is None else lengths.cpu().long().clamp(0, s)
    on = (torch.arange(s)[None, :] < L[:, None]).to(Q.device)[:, None, None, :]  # [B, 1, 1, s]
    q = Q.double()
    k = torch.where(on[:, :, 0, :, None], K.double(), 0.0)
    v = torch.where(on[:, :, 0, :, None], V.double(), 0.0)
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    x = scale * (q @ k.mT)
    ex = abs(scale) * (d + 4) * F * (q.abs() @ k.abs().mT) + E * x.abs()  # what a score is off by: relative error of P
    x = x.masked_fill(~on, -math.inf)
    empty = (L == 0).to(Q.device)[:, None, None]
    lse = torch.logsumexp(x, -1) if s else torch.full((B, heads, n), -math.inf, dtype=torch.float64, device=Q.device)
    P = torch.where(on, (x - torch.where(empty, 0.0, lse)[..., None]).exp(), 0.0)
    H = P @ v
    ex = ex + ex.amax(-1, keepdim=True) if s else ex  # of the weight and of the sum it is divided by
    eP = P * (ex + up + E + (s + 4) * F)
    eH = u * H.abs() + eP @ v.abs() + (s + 4) * F * (P @ v.abs())
    out = {"H": (H, eH), "lse": (lse, torch.where(empty, 0.0, ex.amax(-1) + (s + 4) * F + E * (1 + lse.abs())) if s else lse * 0)}
    if dH is None:
        return out
    g = dH.double()
    dP = g @ v.mT
    D = (g * H).sum(-1, keepdim=True)
    dS = P * (dP - D)
    # D comes from the rounded H; dP and D are sums of d products
    eD = (g.abs() * eH).sum(-1, keepdim=True) + (d + 4) * F * (g.abs() * H.abs()).sum(-1, keepdim=True)
    eS = dS.abs() * (up + ex + E) + P * ((d + 4) * F * (g.abs() @ v.abs().mT) + eD + E * (dP.abs() + D.abs()))
    back = lambda t: t.unflatten(1, (kv, group)).sum(2)  # noqa: E731
    rows = group * n + 4

    def of(value, bound):
        return value, u * value.abs() + bound

    out["dQ"] = of(scale * (dS @ k), abs(scale) * ((eS + (s + 4) * F * dS.abs()) @ k.abs()))
    out["dK"] = of(scale * back(dS.mT @ q), abs(scale) * back((eS + rows * F * dS.abs()).mT @ q.abs()))
    out["dV"] = of(back(P.mT @ g), back((eP + rows * F * P).mT @ g.abs()))
    return out


def rope_angles(theta, positions):
    """theta [axes][pairs] (list), positions [..., axes] -> angles [..., pairs] in 64 bits."""
    return positions.double() @ torch.tensor(theta, dtype=torch.float64, device=positions.device)


def turn(z, angle, magnitude, interleaved):
    """Rows z [B, heads, n, d] in 64 bits turned by angle [B or 1, n, pairs]; the columns behind are passed through."""
    rot = 2 * angle.shape[-1]
    c, s = (magnitude * angle.cos())[:, None], (magnitude * angle.sin())[:, None]
    a, b = (z[..., 0:rot:2], z[..., 1:rot:2]) if interleaved else (z[..., : rot // 2], z[..., rot // 2: rot])
    y = z.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, a * s + b * c
    return y


def pair_size(z, rot, magnitude, interleaved):
    """For each element of z, what its rotated value can be off by per unit of error in the sines: the pair's |a| + |b|."""
    y = z.abs()
    a, b = (z[..., 0:rot:2], z[..., 1:rot:2]) if interleaved else (z[..., : rot // 2], z[..., rot // 2: rot])
    both = abs(magnitude) * (a.abs() + b.abs())
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = both, both
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = both, both
    return y


# an angle is off by pi 2^-24 (its fraction of a turn in fp32) and a sine by a few f more
SINE = 2 * math.pi * F + E


def rope_reference(X, angle, magnitude, interleaved, sign=1):
    x = X.double()
    y = turn(x, sign * angle, magnitude, interleaved)
    return y, half_step(X.dtype) * y.abs() + SINE * pair_size(x, 2 * angle.shape[-1], magnitude, interleaved)


def norm_rope_reference(X, weight, angle, magnitude, eps, interleaved, dY=None):
    """{name: (value, bound)}: Y and, with dY, dX and dw."""
    u, d, rot = half_step(X.dtype), X.shape[-1], 2 * angle.shape[-1]
    x = X.double()
    w = torch.ones(d, dtype=torch.float64, device=X.device) if weight is None else weight.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    z = x * r * w
    y = turn(z, angle, magnitude, interleaved)
    rel = (d + 4) * F + E  # of r, and so of z
    out = {"Y": (y, u * y.abs() + (SINE + rel) * pair_size(z, rot, magnitude, interleaved))}
    if dY is None:
        return out
    g = dY.double()
    dz = turn(g, -angle, magnitude, interleaved)
    edz = SINE * pair_size(g, rot, magnitude, interleaved)
    hat = x * r
    rows = X.shape[0] * X.shape[1] * X.shape[2]
    dw, ab = (dz * hat).sum((0, 1, 2)), (dz * hat).abs().sum((0, 1, 2))
    uw = half_step(weight.dtype) if weight is not None else 0.0
    out["dw"] = (dw, uw * dw.abs() + (edz * hat.abs()).sum((0, 1, 2)) + ((rows + 4) * F + rel) * ab)
    a, ea = dz * w, edz * w.abs()
    m = (a * hat).mean(-1, keepdim=True)
    em = (ea * hat.abs()).mean(-1, keepdim=True) + (2 * rel) * (a * hat).abs().mean(-1, keepdim=True)
    dx = r * (a - hat * m)
    out["dX"] = (dx, u * dx.abs() + r * (ea + hat.abs() * em + 3 * rel * (a.abs() + (hat * m).abs())))
    return out


def assert_within(got, reference, what):
    value, bound = reference
    assert tuple(got.shape) == tuple(value.shape), (what, got.shape, value.shape)
    g = got.double()
    same = g == value  # infinities too
    off = (g - value).abs()
    bad = ~(same | (off <= bound + 1e-30))
    if bool(bad.any()):
        at = torch.nonzero(bad)[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; at {at}: got {float(g[i])!r}, "
                             f"reference {float(value[i])!r}, bound {float(bound[i]):.3e}")
