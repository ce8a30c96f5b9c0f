"""Cross attention, rotary positions and normalised rotary queries and keys: the calls that are timed.

`listed()` and `draw()` give cases, `prepare()` the tensors a program has in hand, `run()` one pass through an operator
(in plain torch, or, with `own` set, through this package), `exact()` the same results in 64 bits."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def cross(name, B, heads, kv, n, s, d, dtype="bf16", train=False, ragged=False, tokens=False):
    """heads query heads over kv key heads, n queries, s encoder states; ragged: each batch entry has a length of its
    own; tokens: the tensors are views of token-major projections [B, n, heads, d]."""
    return {"name": name, "op": "cross", "B": B, "heads": heads, "kv": kv, "n": n, "s": s, "d": d, "dtype": dtype,
            "train": train, "ragged": ragged, "tokens": tokens}


def norm_rope(name, B, heads, kv, n, d, rot, dtype="bf16", train=False, interleaved=False, tokens=False, grid=0):
    """grid: columns of an image grid whose rows and columns are the two axes of the positions (0: one axis)."""
    return {"name": name, "op": "norm_rope", "B": B, "heads": heads, "kv": kv, "n": n, "d": d, "rot": rot, "dtype": dtype,
            "train": train, "interleaved": interleaved, "tokens": tokens, "grid": grid, "far": 0, "scaling": "none"}


def rope(name, B, heads, n, d, rot, dtype="bf16", train=False, interleaved=False, tokens=False, far=0, scaling="none"):
    """far: the positions start here; scaling: how the frequencies are stretched for long contexts."""
    return {"name": name, "op": "rope", "B": B, "heads": heads, "kv": 0, "n": n, "d": d, "rot": rot, "dtype": dtype,
            "train": train, "interleaved": interleaved, "tokens": tokens, "grid": 0, "far": far, "scaling": scaling}


def listed():
    return [
        # a long image sequence attends to a long encoder's states: the largest, bound by the products
        cross("cross_long", 2, 16, 16, 16384, 4096, 128),
        # training step of a detection layer: 50 x 84 patches over a text encoder's padded batch
        cross("cross_train_det", 8, 12, 12, 4200, 1000, 64, train=True, ragged=True),
        # classification batch over short prompts, padded
        cross("cross_deit", 256, 12, 12, 197, 77, 64, ragged=True),
        # training step with shared key heads and token-major projections
        cross("cross_train_shared", 2, 16, 4, 2049, 1500, 128, train=True, tokens=True),
        # serving: one token of 64 requests over their encoders' states, shared key heads
        cross("cross_step", 64, 32, 8, 1, 8192, 128, ragged=True),
        # serving: one token of one request: latency
        cross("cross_step_one", 1, 12, 12, 1, 1500, 64),
        # fp32 training step of a small model
        cross("cross_train_f32", 4, 6, 6, 197, 300, 64, dtype="f32", train=True, ragged=True),
        # queries and keys of a long sequence out of token-major projections
        norm_rope("norm_rope_long", 4, 16, 16, 16384, 128, 128, tokens=True),
        # training step on image-grid positions
        norm_rope("norm_rope_train_det", 8, 12, 12, 4200, 64, 64, train=True, grid=84),
        # serving: one token of 64 requests
        norm_rope("norm_rope_step", 64, 32, 8, 1, 128, 128, tokens=True),
        # far positions of a stretched context, half of each head rotated
        rope("rope_far", 1, 32, 32768, 128, 64, interleaved=True, tokens=True, far=900000, scaling="bands"),
        # fp32 training step, a part of the head in halves
        rope("rope_train_f32", 4, 6, 1000, 64, 32, dtype="f32", train=True, scaling="linear"),
    ]


def spread(rng, low, high):
    """A whole number between low and high, even in its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    kind = rng.choice(("cross", "cross", "step", "norm_rope", "rope"))
    d, dtype, train = rng.choice((64, 64, 128, 128, 32, 16)), rng.choice(("bf16", "bf16", "bf16", "f32")), rng.random() < 0.4
    kv = rng.choice((1, 2, 3, 4, 8, 12))
    heads = kv * rng.choice((1, 1, 2, 4))
    tokens = rng.random() < 0.5
    if kind == "cross":
        n, s = spread(rng, 2, 16384), spread(rng, 8 if train else 1, 8192)
        # f32 and training cases are smaller, so that none costs more than the largest listed one
        most = (1 << 31 if dtype == "bf16" else 1 << 28) // (4 if train else 1)
        while heads * n * s > most:
            n, s = max(2, n * 2 // 3), max(8, s * 3 // 4)
        B = spread(rng, 1, max(1, min(64, most // (heads * n * s), (1 << 26) // (heads * (n + s) * d))))
        return unnamed(cross("", B, heads, kv, n, s, d, dtype, train, rng.random() < 0.5, tokens))
    if kind == "step":
        s = spread(rng, 1, 65536)
        B = spread(rng, 1, max(1, min(128, (1 << 27) // (s * kv * d))))
        return unnamed(cross("", B, heads, kv, rng.choice((1, 1, 1, 2, 5)), s, d, dtype, False, rng.random() < 0.5, tokens))
    n = spread(rng, 1, 32768)
    while n * 2 * heads * d > 1 << 26:
        n = n * 2 // 3
    B = spread(rng, 1, max(1, min(64, (1 << 26) // (n * 2 * heads * d))))
    rot = rng.choice((d, d, d // 2, max(2, d // 4), max(2, d // 16 * 6)))
    if kind == "rope":
        return unnamed(rope("", B, heads, n, d, rot, dtype, train, rng.random() < 0.5, tokens, rng.choice((0, 0, 5000, 1000000)),
                            rng.choice(("none", "linear", "base", "bands"))))
    grid = spread(rng, 2, 200) if rot % 4 == 0 and rng.random() < 0.4 else 0
    return unnamed(norm_rope("", B, heads, kv, n, d, rot, dtype, train, rng.random() < 0.5, tokens, grid))


def frequencies(c):
    """Radians that one position adds to each pair's angle, [axes, rot / 2] in 64 bits, and the factor on the rotated part."""
    if c["grid"]:  # rows turn the first half of the pairs, columns the second
        half = c["rot"] // 4
        theta = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        none = torch.zeros_like(theta)
        return torch.stack([torch.cat([theta, none]), torch.cat([none, theta])]), 1.0
    pairs = c["rot"] // 2
    k = torch.arange(pairs, dtype=torch.float64) / pairs
    theta, factor, original = 10000.0 ** -k, 8.0, 131072
    if c["scaling"] == "linear":
        return (theta / factor)[None], 1.0
    if c["scaling"] == "base":
        return ((10000.0 * factor ** (pairs / max(1, pairs - 1))) ** -k)[None], 1.0
    if c["scaling"] == "bands":  # fast pairs stay, slow ones are divided, between 1 and 32 turns a mixture
        keep = ((original * theta / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        return (theta * keep + theta / factor * (1 - keep))[None], 0.1 * math.log(factor) + 1.0
    return theta[None], 1.0


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(B, heads, n, gain=1.0):
        shape = (B, n, heads, c["d"]) if c["tokens"] else (B, heads, n, c["d"])
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(gain).to(dt)
        return x.transpose(1, 2) if c["tokens"] else x

    st = {"case": c}
    if c["op"] == "cross":
        # scores of spread about 1.5: some states weigh more than others, none alone
        st["Q"], st["K"] = normal(c["B"], c["heads"], c["n"], 1.5), normal(c["B"], c["kv"], c["s"])
        st["V"] = normal(c["B"], c["kv"], c["s"])
        st["lengths"] = None
        if c["ragged"]:
            # short ones may be empty in serving; a training batch has two states at least
            least = c["s"] // 4 if c["s"] >= 100 else 2 if c["train"] else 0
            st["lengths"] = torch.randint(least, c["s"] + 1, (c["B"],), generator=g, device=dev, dtype=torch.int32)
        if c["train"]:
            st["dH"] = normal(c["B"], c["heads"], c["n"])
        st["scale"] = c["d"] ** -0.5
        return st
    theta, st["magnitude"] = frequencies(c)
    st["theta"] = theta.to(dev)
    # the same angles as 64-bit fractions of a turn, two's complement
    turns = [[int(round(t / (2 * math.pi) * 2 ** 64)) % 2 ** 64 for t in row] for row in theta.tolist()]
    st["phases"] = torch.tensor([[t - 2 ** 64 if t >= 2 ** 63 else t for t in row] for row in turns], dtype=torch.int64).to(dev)
    i = torch.arange(c["n"], device=dev, dtype=torch.int32)
    if c["grid"]:
        st["positions"] = torch.stack([i // c["grid"], i % c["grid"]], -1).contiguous()
    else:  # every entry is at a place of its own
        st["positions"] = c["far"] + i[None, :] + torch.randint(0, 1000, (c["B"], 1), generator=g, device=dev, dtype=torch.int32)
    names = (("Q", "heads"), ("K", "kv")) if c["op"] == "norm_rope" else (("Q", "heads"),)
    for name, heads in names:
        st[name] = normal(c["B"], c[heads], c["n"], 2.0 if c["op"] == "norm_rope" else 1.0)
        if c["train"]:
            st["d" + name] = normal(c["B"], c[heads], c["n"])
        if c["op"] == "norm_rope":
            st["w" + name] = (1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt)
    return st


# ---------------------------------------------------------------------- plain forms

def plain_cross(st):
    c = st["case"]
    B, kv, group, n, s, d = c["B"], c["kv"], c["heads"] // c["kv"], c["n"], c["s"], c["d"]
    q = st["Q"].float().reshape(B, kv, group * n, d)
    k, v = st["K"].float(), st["V"].float()
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"])
    if st["lengths"] is not None:
        out = torch.arange(s, device=q.device)[None, :] >= st["lengths"][:, None]
        x.masked_fill_(out[:, None, None, :], -math.inf)
        v = v.masked_fill(out[:, None, :, None], 0)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total.clamp(min=1e-30))
    h = torch.matmul(p, v)
    H = h.reshape(B, kv * group, n, d).to(st["Q"].dtype)
    if not c["train"]:
        return {"H": H}
    lse = (top + total.log()).reshape(B, kv * group, n)
    dh = st["dH"].float().reshape(B, kv, group * n, d)
    dv = torch.matmul(p.transpose(-1, -2), dh)
    ds = torch.matmul(dh, v.transpose(-1, -2)).sub_((dh * h).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k).mul_(st["scale"]).reshape(B, kv * group, n, d)
    dk = torch.matmul(ds.transpose(-1, -2), q).mul_(st["scale"])
    dt = H.dtype
    return {"H": H, "lse": lse, "dQ": dq.to(dt), "dK": dk.to(dt), "dV": dv.to(dt)}


def plain_angles(st):
    pos = st["positions"].double()
    t = torch.matmul(pos, st["theta"])[None] if st["case"]["grid"] else pos[..., None] * st["theta"][0]
    return (t.cos() * st["magnitude"]).float()[:, None], (t.sin() * st["magnitude"]).float()[:, None]


def plain_turn(x, cos, sin, rot, interleaved):
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, a * sin + b * cos
    return y


EPS = 1e-6


def plain_norm_rope_one(c, x, w, dy, cos, sin):
    x32, w32 = x.float(), w.float()
    r = (x32.square().mean(-1, keepdim=True) + EPS).rsqrt()
    hat = x32 * r
    y = plain_turn(hat * w32, cos, sin, c["rot"], c["interleaved"]).to(x.dtype)
    if dy is None:
        return y, None, None
    dz = plain_turn(dy.float(), cos, -sin, c["rot"], c["interleaved"])
    dw = (dz * hat).sum((0, 1, 2))
    dz = dz * w32
    dx = r * (dz - hat * (dz * hat).mean(-1, keepdim=True))
    return y, dx.to(x.dtype), dw.to(w.dtype)


def plain_rope(st):
    c = st["case"]
    cos, sin = plain_angles(st)
    if c["op"] == "norm_rope":
        q, dq, dwq = plain_norm_rope_one(c, st["Q"], st["wQ"], st.get("dQ"), cos, sin)
        k, dk, dwk = plain_norm_rope_one(c, st["K"], st["wK"], st.get("dK"), cos, sin)
        return {"Q": q, "K": k, "dQ": dq, "dK": dk, "dwQ": dwq, "dwK": dwk} if c["train"] else {"Q": q, "K": k}
    out = {"X": plain_turn(st["Q"].float(), cos, sin, c["rot"], c["interleaved"]).to(st["Q"].dtype)}
    if c["train"]:
        out["dX"] = plain_turn(st["dQ"].float(), cos, -sin, c["rot"], c["interleaved"]).to(st["Q"].dtype)
    return out


# ---------------------------------------------------------------------- the package's own calls

def own_cross(st):
    import linear_complexity_anchor_gb300 as aa
    if not st["case"]["train"]:
        return {"H": aa.cross_forward(st["Q"], st["K"], st["V"], st["lengths"], scale=st["scale"])}
    H, lse = aa.cross_forward(st["Q"], st["K"], st["V"], st["lengths"], scale=st["scale"], return_lse=True)
    dQ, dK, dV = aa.cross_backward(st["Q"], st["K"], st["V"], H, lse, st["dH"], st["lengths"], scale=st["scale"])
    return {"H": H, "lse": lse, "dQ": dQ, "dK": dK, "dV": dV}


def own_rope(st):
    import linear_complexity_anchor_gb300 as aa
    c, table, pos = st["case"], (st["phases"], st["magnitude"]), st["positions"]
    if c["op"] == "rope":
        out = {"X": aa.rope(st["Q"], table, pos, interleaved=c["interleaved"])}
        if c["train"]:
            out["dX"] = aa.rope_backward(st["dQ"], table, pos, interleaved=c["interleaved"])
        return out
    how = {"q_weight": st["wQ"], "k_weight": st["wK"], "q_positions": pos, "k_positions": pos, "eps": EPS, "interleaved": c["interleaved"]}
    Q, K = aa.norm_rope(st["Q"], st["K"], table, **how)
    if not c["train"]:
        return {"Q": Q, "K": K}
    dQ, dK, dwQ, dwK = aa.norm_rope_backward(st["Q"], st["K"], st["dQ"], st["dK"], table, **how)
    return {"Q": Q, "K": K, "dQ": dQ, "dK": dK, "dwQ": dwQ, "dwK": dwK}


def run(state):
    if state["case"]["op"] == "cross":
        return own_cross(state) if own else plain_cross(state)
    return own_rope(state) if own else plain_rope(state)


# ---------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "cross":
        share = (0.5 if c["s"] < 100 else 0.625) if c["ragged"] else 1.0  # the mean length over s
        q, kv = c["B"] * c["heads"] * c["n"] * c["d"], c["B"] * c["kv"] * c["s"] * c["d"] * share
        pairs = c["B"] * c["heads"] * c["n"] * c["s"] * share
        # forward: Q, K, V in, H out; a training step: dH in, dQ, dK, dV out too, and lse
        moved = (4 * q + 4 * kv) * size + 4 * q / c["d"] if c["train"] else (2 * q + 2 * kv) * size
        return {"bytes": moved, "flops": pairs * c["d"] * (14 if c["train"] else 4)}
    x = c["B"] * (c["heads"] + c["kv"]) * c["n"] * c["d"]
    each = 4 if c["train"] else 2  # x in, y out; a training step: dy in, dx out too
    return {"bytes": each * x * size, "flops": x * (6 if c["op"] == "rope" else 10) * (2 if c["train"] else 1)}


# ---------------------------------------------------------------------- in 64 bits, from the definitions

def exact_cross(st):
    c = st["case"]
    group = c["heads"] // c["kv"]
    B, n, d = c["B"], c["n"], c["d"]
    keys = ("H", "lse", "dQ", "dK", "dV") if c["train"] else ("H",)
    dev = st["Q"].device
    out = {"H": torch.zeros(B, c["heads"], n, d, dtype=torch.float64, device=dev)}
    if c["train"]:
        out["lse"] = torch.full((B, c["heads"], n), -math.inf, dtype=torch.float64, device=dev)
        out["dQ"] = torch.zeros_like(out["H"])
        out["dK"] = torch.zeros(B, c["kv"], c["s"], d, dtype=torch.float64, device=dev)
        out["dV"] = torch.zeros_like(out["dK"])
    lengths = [c["s"]] * B if st["lengths"] is None else st["lengths"].tolist()
    for b, L in enumerate(lengths):
        if L == 0:
            continue
        if c["heads"] * n * L <= 1 << 26:  # all heads of an entry at once
            parts = [slice(0, c["kv"])]
        else:
            parts = [slice(h, h + 1) for h in range(c["kv"])]
        for kvs in parts:
            hs = slice(kvs.start * group, kvs.stop * group)
            q = st["Q"][b, hs].double().unflatten(0, (-1, group))
            k, v = st["K"][b, kvs, :L].double()[:, None], st["V"][b, kvs, :L].double()[:, None]
            x = st["scale"] * (q @ k.mT)
            lse = torch.logsumexp(x, -1)
            p = (x - lse[..., None]).exp()
            h = p @ v
            out["H"][b, hs] = h.flatten(0, 1)
            if c["train"]:
                dh = st["dH"][b, hs].double().unflatten(0, (-1, group))
                dp = dh @ v.mT
                ds = p * (dp - (dp * p).sum(-1, keepdim=True))
                out["lse"][b, hs] = lse.flatten(0, 1)
                out["dQ"][b, hs] = st["scale"] * (ds @ k).flatten(0, 1)
                out["dK"][b, kvs, :L] = st["scale"] * (ds.mT @ q).sum(1)
                out["dV"][b, kvs, :L] = (p.mT @ dh).sum(1)
    return {k: out[k] for k in keys}


def exact_one(c, angle, g, x, w, dy):
    """x [n, d] or more in front: complex numbers turned by the angle, the rest of the head as it is."""
    def turn(z, sign):
        r = z[..., : c["rot"]]
        r = r.unflatten(-1, (-1, 2)) if c["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
        r = torch.view_as_complex(r.contiguous()) * torch.polar(torch.full_like(angle, g), sign * angle)
        r = torch.view_as_real(r)
        r = r.flatten(-2) if c["interleaved"] else r.transpose(-1, -2).flatten(-2)
        return torch.cat([r, z[..., c["rot"]:]], -1)

    x = x.double()
    if w is None:
        return turn(x, 1), None if dy is None else turn(dy.double(), -1), None
    size = ((x * x).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
    y = turn(x / size * w.double(), 1)
    if dy is None:
        return y, None, None
    dz = turn(dy.double(), -1)
    dw = (dz * x / size).flatten(0, -2).sum(0)
    a = dz * w.double() / size
    return y, a - x * (a * x).sum(-1, keepdim=True) / (c["d"] * size * size), dw


def exact_rope(st):
    c = st["case"]
    pos = st["positions"].double()
    if c["grid"]:
        angle = (pos[:, 0, None] * st["theta"][0] + pos[:, 1, None] * st["theta"][1])[None, None]
    else:
        angle = (pos[:, :, None] * st["theta"][0])[:, None]
    if c["op"] == "rope":
        y, dx, _ = exact_one(c, angle, st["magnitude"], st["Q"], None, st.get("dQ"))
        return {"X": y, "dX": dx} if c["train"] else {"X": y}
    q, dq, dwq = exact_one(c, angle, st["magnitude"], st["Q"], st["wQ"], st.get("dQ"))
    k, dk, dwk = exact_one(c, angle, st["magnitude"], st["K"], st["wK"], st.get("dK"))
    return {"Q": q, "K": k, "dQ": dq, "dK": dk, "dwQ": dwq, "dwK": dwk} if c["train"] else {"Q": q, "K": k}


def exact(case, seed):
    st = prepare(case, seed)
    return exact_cross(st) if case["op"] == "cross" else exact_rope(st)
