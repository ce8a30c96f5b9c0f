"""64-bit references of attention with decaying states and of the norm of a residual sum, each with a bound on what the
roundings of the kernels can add up to, element by element (notation of tests/ops_reference.py)."""
import torch

from tests.ops_reference import E, F, half_step


def rates(log_decay):
    return log_decay.double().clamp(-1e4, 0)


def powers(log_decay, k):
    """exp(log_decay)^k for whole k >= 0, 0 for negative ones: [heads, *k.shape]."""
    k = k.double()
    return torch.where(k < 0, 0.0, (rates(log_decay).view(-1, *[1] * k.dim()) * k.clamp(min=0)).exp())


def lengths_of(lengths, B, n, device):
    return torch.full((B,), n, device=device) if lengths is None else lengths.long().clamp(0, n)


def decay_reference(Q, K, V, log_decay, lengths, state, scale, dH=None, dlast=None):
    """{name: (value, bound)}: H and last; with dH also dQ, dK, dV and (with a state) dstate.

    bf16: a pair's weight meets c as bf16, and the state meets a as bf16 (u each, of the magnitudes they are summed
    over: never more than u sum |weight| |c| over all pairs, with |weight| = g^(i-j) |a| . |b| for those that go by the
    state); the rows that are added to a state are two bf16 numbers, exact to 2^-17.  A sum of fp32 numbers as
    there; the factors g^k are carried over n / 64 chunks, each with a rounding or two, and exp's."""
    u = half_step(Q.dtype)
    bf16 = Q.dtype == torch.bfloat16
    B, heads, n, d = Q.shape
    L = lengths_of(lengths, B, n, Q.device)
    i = torch.arange(n, device=Q.device)
    on = (i[None] < L[:, None])[:, None, :, None]
    q, k, v = (torch.where(on, x.double(), 0.0) for x in (Q, K, V))
    pair = powers(log_decay, i[:, None] - i[None])                                  # [heads, n, n]
    ahead = powers(log_decay, i + 1)[None, ..., None]                               # g^(i + 1)
    rest = powers(log_decay, L[:, None] - 1 - i[None]).transpose(0, 1)[..., None]   # g^(L - 1 - j), [B, heads, n, 1]
    whole = powers(log_decay, L).transpose(0, 1)[..., None, None]
    X = torch.zeros(B, heads, d, d, dtype=torch.float64, device=Q.device) if state is None else state.double()
    sums = (n + 3 * d + 64) * F + E + (2.0 ** -16 if bf16 else 0.0)                  # of what is summed over rows
    fine = (n + 3 * d + 64) * F + E

    def outer(a, b):
        return a.mT @ b

    def one(a, b, c, w, X, p, s):
        """o = p (w_ij a_i . b_j) c_j + s a_i X_i, X_i given as (factor of row i, matrix); and its bound"""
        f, M = X
        x = p * (a @ b.mT) * w
        o = x @ c + s * f * (a @ M)
        mag = abs(p) * ((a.abs() @ b.abs().mT) * w) @ c.abs() + abs(s) * f * (a.abs() @ M.abs())
        # where pairs go by themselves (a chunk of 128 or less) their weights are rounded, else |a| |state|
        near = (i[:, None] // 128 == i[None] // 128)
        m = (x.abs() * near) @ c.abs() + abs(p) * ((a.abs() @ b.abs().mT) * w * ~near) @ c.abs() + abs(s) * f * (a.abs() @ M.abs())
        return o, u * o.abs() + (2 * u * m if bf16 else 0.0) + sums * mag

    keep = lambda t: tuple(torch.where(on, x, 0.0) for x in t)  # noqa: E731
    out = {"H": keep(one(q, k, v, pair, (ahead, X), scale, scale))}
    last = outer(k * rest, v) + whole * X
    out["last"] = (last, sums * outer(k.abs() * rest, v.abs()) + fine * whole * X.abs())
    if dH is None:
        return out
    dh = torch.where(on, dH.double(), 0.0)
    G = torch.zeros_like(X) if dlast is None else dlast.double()
    out["dQ"] = keep(one(dh, v, k, pair, (ahead, X.mT), scale, scale))
    out["dK"] = keep(one(v, dh, q, pair.mT, (rest, G.mT), scale, 1.0))
    out["dV"] = keep(one(k, q, dh, pair.mT, (rest, G), scale, 1.0))
    if state is not None:
        dstate = scale * outer(q * ahead, dh) + whole * G
        out["dstate"] = (dstate, abs(scale) * sums * outer(q.abs() * ahead, dh.abs()) + fine * whole * G.abs() + F * dstate.abs())
    return out


def sum_of(X, R):
    return X if R is None else (X.float() + R.float()).to(X.dtype)


def add_norm_reference(X, R, weight, eps):
    """(S as it is kept, (Y in 64 bits, what fp32 arithmetic may be off by))"""
    S = sum_of(X, R)
    s, D = S.double(), X.shape[-1]
    w = torch.ones(D, dtype=torch.float64, device=X.device) if weight is None else weight.double()
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * w
    return S, (y, ((D + 4) * F + E) * y.abs())


def add_norm_backward_reference(S, dY, weight, dS, eps):
    """{name: (value, bound)}: dX and dweight."""
    u, D = half_step(S.dtype), S.shape[-1]
    s, g = S.double(), dY.double()
    w = torch.ones(D, dtype=torch.float64, device=S.device) if weight is None else weight.double()
    r = 1 / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    hat, rel = s * r, (D + 4) * F + E
    rows = S.numel() // D
    dw, ab = (g * hat).reshape(-1, D).sum(0), (g * hat).abs().reshape(-1, D).sum(0)
    uw = half_step(weight.dtype) if weight is not None else 0.0
    a = g * w
    m, em = (a * hat).mean(-1, keepdim=True), 2 * rel * (a * hat).abs().mean(-1, keepdim=True)
    dx = r * (a - hat * m)
    ex = r * (hat.abs() * em + 3 * rel * (a.abs() + (hat * m).abs()))
    if dS is not None:
        ex, dx = ex + F * (dx.abs() + dS.double().abs()), dx + dS.double()
    return {"dX": (dx, u * dx.abs() + ex), "dweight": (dw, uw * dw.abs() + ((rows + 4) * F + rel) * ab)}
