"""Attention with decaying states, and the norm of a residual sum: the calls that are timed.

`listed()` and `draw()` give cases, `prepare()` the tensors a program has in hand, `run()` one pass through an operator
(in plain torch, or, with `own` set, through this package), `exact()` the same results in 64 bits."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
TOP = 448.0  # the largest 8-bit value


def decay(name, B, heads, n, d, dtype="bf16", train=False, ragged=False, tokens=False, state=False):
    """n tokens of `heads` heads of d; ragged: each batch entry has a length of its own; tokens: the tensors are views
    of token-major projections [B, n, heads, d]; state: the entries begin with a state (and, in training, get a
    gradient of the last one). The last state is returned too."""
    return {"name": name, "op": "decay", "B": B, "heads": heads, "n": n, "d": d, "dtype": dtype, "train": train,
            "ragged": ragged, "tokens": tokens, "state": state}


def step(name, B, heads, d, n=1, dtype="bf16", pool=0):
    """n tokens of B requests, whose states are those of `pool` slots (0: one slot a request, in order)."""
    return {"name": name, "op": "step", "B": B, "heads": heads, "n": n, "d": d, "dtype": dtype, "pool": pool}


def norm(name, rows, D, dtype="bf16", bits8=False, group=0, train=False, residual=True):
    """rows of D columns; bits8: the result in 8 bits, with a scale for each `group` of columns (0: for each row)."""
    return {"name": name, "op": "norm", "rows": rows, "D": D, "dtype": dtype, "bits8": bits8, "group": group,
            "train": train, "residual": residual}


def listed():
    return [
        # the prompts of four long documents: the largest, bound by memory
        decay("decay_long", 4, 16, 16384, 128),
        # training step of a detection layer: 50 x 84 patches, padded
        decay("decay_train_det", 8, 12, 4200, 64, train=True, ragged=True),
        # training step of a long text, token-major projections
        decay("decay_train_tokens", 2, 16, 8192, 128, train=True, tokens=True),
        # classification batch: many short sequences, padded
        decay("decay_deit", 128, 12, 197, 64, ragged=True),
        # serving: the next part of one request's prompt
        decay("decay_prompt_one", 1, 16, 2049, 128, tokens=True, state=True),
        # fp32 training step of a small model, whose sequences go on from the ones before
        decay("decay_train_f32", 4, 6, 197, 64, dtype="f32", train=True, ragged=True, state=True),
        # serving: one token of 64 requests, whose states lie in a pool
        step("decay_step", 64, 32, 128, pool=100),
        # serving: one token of one request: latency
        step("decay_step_one", 1, 12, 64),
        # prompts: the residual's addition, the norm, and 8 bits for the products behind it
        norm("norm_8bit_long", 65536, 2048, bits8=True),
        # classification batch, a scale for each 128 columns
        norm("norm_8bit_deit", 128 * 197, 768, bits8=True, group=128),
        # serving: one token of 64 requests
        norm("norm_8bit_step", 64, 4096, bits8=True, group=128),
        # training step of a detection layer
        norm("norm_train_det", 8 * 4200, 768, train=True),
    ]


def spread(rng, low, high):
    """A whole number between low and high, even in its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    kind = rng.choice(("decay", "decay", "decay", "step", "norm", "norm"))
    dtype, train = rng.choice(("bf16", "bf16", "bf16", "f32")), rng.random() < 0.5
    d = rng.choice((64, 64, 128, 128, 32, 16))
    if kind == "decay":
        n, heads = spread(rng, 1, 32768), rng.choice((1, 2, 3, 6, 12, 16, 32))
        # f32 and training cases are smaller, so that none costs more than the largest listed one
        most = (1 << 27 if dtype == "bf16" else 1 << 24) // (4 if train else 1)
        while heads * n * d > most:
            n = n * 2 // 3
        B = spread(rng, 1, max(1, min(128, most // (heads * n * d), (1 << 25) // (heads * d * d))))
        return unnamed(decay("", B, heads, n, d, dtype, train, rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.4))
    if kind == "step":
        heads = rng.choice((1, 3, 8, 12, 16, 32))
        B = spread(rng, 1, max(1, min(256, (1 << 26) // (heads * d * d))))
        return unnamed(step("", B, heads, d, rng.choice((1, 1, 1, 2, 4)), dtype, rng.choice((0, B + spread(rng, 1, 64)))))
    D = 16 * spread(rng, 1, 1024)
    rows = spread(rng, 1, max(1, min(200000, (1 << 27) // D // (1 if dtype == "bf16" else 2) // (2 if train else 1))))
    bits8 = not train and rng.random() < 0.7
    return unnamed(norm("", rows, D, dtype, bits8, rng.choice((0, 0, 128, 64, 32)) if bits8 else 0, train, rng.random() < 0.8))


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    st = {"case": c}
    if c["op"] == "norm":
        st["X"] = normal(c["rows"], c["D"]).to(dt)
        # a residual stream has grown over the layers, a few of its columns more than the others
        big = 1 + 9 * (torch.rand(c["D"], generator=g, device=dev) < 0.01)
        st["R"] = (normal(c["rows"], c["D"]) * 3 * big).to(dt) if c["residual"] else None
        st["w"] = (1 + 0.2 * normal(c["D"])).to(dt)
        if c["train"]:
            st["dY"], st["dS"] = normal(c["rows"], c["D"]).to(dt), normal(c["rows"], c["D"]).to(dt)
        return st
    B, heads, n, d = c["B"], c["heads"], c["n"], c["d"]

    def rows():
        if c.get("tokens"):
            return normal(B, n, heads, d).to(dt).transpose(1, 2)
        return normal(B, heads, n, d).to(dt)

    for name in "QKV":
        st[name] = rows()
    # a head keeps the last 30 to 4000 tokens
    reach = 5 + 7 * (torch.arange(heads, device=dev) + torch.rand(heads, generator=g, device=dev)) / heads
    st["log_decay"] = torch.log1p(-torch.exp2(-reach.double())).float()
    st["scale"] = d ** -0.5
    if c["op"] == "step":
        pool = c["pool"] or B
        st["states"] = normal(pool, heads, d, d) * 5
        st["slots"] = torch.randperm(pool, generator=g, device=dev)[:B].to(torch.int32) if c["pool"] else None
        return st
    st["lengths"] = torch.randint(n // 4, n + 1, (B,), generator=g, device=dev, dtype=torch.int32) if c["ragged"] else None
    st["state"] = normal(B, heads, d, d) * 5 if c["state"] else None
    if c["train"]:
        st["dH"] = rows()
        st["dstate"] = normal(B, heads, d, d) * 0.1 if c["state"] else None
    return st


# ---------------------------------------------------------------------- plain forms

CHUNK = 128


def powers(log_decay, k):
    """decay^k for whole numbers k >= 0 (0 for negative ones), [heads, *k.shape]: the exponents in 64 bits."""
    k = k.double()
    x = log_decay.double().view(-1, *([1] * k.dim())) * k.clamp(min=0)
    return torch.where(k < 0, 0.0, x.exp()).float()


def plain_pass(a, b, c, log_decay, state):
    """o_i = sum_{j <= i} decay^(i - j) (a_i . b_j) c_j + decay^(i + 1) a_i state, by chunks whose states are summed by
    one product; all fp32 [B, heads, n, d]."""
    B, heads, n, d = a.shape
    size = min(CHUNK, n)
    chunks = -(-n // size)
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, chunks * size - n)).reshape(B, heads, chunks, size, d) for x in (a, b, c))
    i = torch.arange(size, device=a.device)
    x = torch.matmul(a, b.transpose(-1, -2)).mul_(powers(log_decay, i[:, None] - i[None, :])[:, None])
    o = torch.matmul(x, c)
    if chunks > 1 or state is not None:
        own_states = torch.matmul((b * powers(log_decay, size - 1 - i)[:, None, :, None]).transpose(-1, -2), c)
        k = torch.arange(chunks, device=a.device)
        before = torch.where(k[:, None] > k[None, :], size * (k[:, None] - 1 - k[None, :]), -1)
        states = torch.matmul(powers(log_decay, before), own_states.flatten(-2))
        if state is not None:
            states += powers(log_decay, k * size)[:, :, None] * state.flatten(-2)[:, :, None]
        a = a * powers(log_decay, i + 1)[:, None, :, None]
        o += torch.matmul(a, states.unflatten(-1, (d, d)))
    return o.reshape(B, heads, chunks * size, d)[:, :, :n]


def plain_decay(st):
    c = st["case"]
    n, g, dt, scale = c["n"], st["log_decay"], st["Q"].dtype, st["scale"]
    q, k, v = (st[x].float() for x in "QKV")
    i = torch.arange(n, device=q.device)
    L = torch.full((c["B"],), n, device=q.device) if st["lengths"] is None else st["lengths"].long()
    on = i[None, :] < L[:, None]
    q, k, v = (x.masked_fill(~on[:, None, :, None], 0) for x in (q, k, v))
    state = st["state"]
    rest = powers(g, L[:, None] - 1 - i[None, :]).transpose(0, 1)[..., None]  # decay^(L - 1 - j), [B, heads, n, 1]
    whole = powers(g, L).transpose(0, 1)[..., None, None]                      # decay^L
    last = torch.matmul((k * rest).transpose(-1, -2), v)
    if state is not None:
        last += whole * state
    h = plain_pass(q * scale, k, v, g, state).masked_fill_(~on[:, None, :, None], 0)
    out = {"H": h.to(dt), "state": last}
    if not c["train"]:
        return out
    dh, ds = st["dH"].float().masked_fill(~on[:, None, :, None], 0), st["dstate"]
    dq = plain_pass(dh * scale, v, k, g, None if state is None else state.transpose(-1, -2)).masked_fill_(~on[:, None, :, None], 0)
    back = lambda x: x.flip(2)  # noqa: E731
    dk = back(plain_pass(back(v) * scale, back(dh), back(q), g, None)) * on[:, None, :, None]
    dv = back(plain_pass(back(k) * scale, back(q), back(dh), g, None)) * on[:, None, :, None]
    if ds is not None:
        dk += rest * torch.matmul(v, ds.transpose(-1, -2))
        dv += rest * torch.matmul(k, ds)
    out |= {"dQ": dq.to(dt), "dK": dk.to(dt), "dV": dv.to(dt)}
    if state is not None:
        out["dstate"] = whole * ds + scale * torch.matmul((q * powers(g, i + 1)[None, ..., None]).transpose(-1, -2), dh)
    return out


def plain_step(st):
    """The tokens together: the state before them, and what each adds for itself and the later ones."""
    c = st["case"]
    n, g = c["n"], st["log_decay"]
    q, k, v = (st[x].float() for x in "QKV")
    s = st["states"] if st["slots"] is None else st["states"][st["slots"].long()]
    h = plain_pass(q * st["scale"], k, v, g, s)
    i = torch.arange(n, device=q.device)
    new = s * powers(g, torch.tensor([n], device=q.device))[None, :, :, None]
    new += torch.matmul((k * powers(g, n - 1 - i)[None, ..., None]).transpose(-1, -2), v)
    if st["slots"] is None:
        st["states"].copy_(new)
    else:
        st["states"].index_copy_(0, st["slots"].long(), new)
    return {"H": h.to(st["Q"].dtype), "states": st["states"]}


def plain_norm(st):
    c = st["case"]
    dt = st["X"].dtype
    s = st["X"] if st["R"] is None else (st["X"].float() + st["R"].float()).to(dt)
    x, w = s.float(), st["w"].float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    hat = x * r
    y = hat * w
    out = {} if st["R"] is None else {"S": s}
    if c["bits8"]:
        size = c["group"] or c["D"]
        groups = -(-c["D"] // size)
        z = torch.nn.functional.pad(y, (0, groups * size - c["D"])).unflatten(-1, (groups, size))
        scales = z.abs().amax(-1) / TOP
        z = z / scales.masked_fill(scales == 0, 1)[..., None]
        return out | {"Y": z.clamp(-TOP, TOP).flatten(-2)[:, : c["D"]].to(torch.float8_e4m3fn), "scales": scales}
    out["Y"] = y.to(dt)
    if c["train"]:
        dy = st["dY"].float()
        dw = (dy * hat).sum(0)
        dy = dy * w
        out["dX"] = (r * (dy - hat * (dy * hat).mean(-1, keepdim=True)) + st["dS"].float()).to(dt)
        out["dw"] = dw.to(dt)
    return out


# ---------------------------------------------------------------------- the package's own calls

def own_decay(st):
    import linear_complexity_anchor_gb300 as aa
    how = {"lengths": st["lengths"], "state": st["state"], "scale": st["scale"]}
    H, state = aa.decay_forward(st["Q"], st["K"], st["V"], st["log_decay"], return_state=True, **how)
    out = {"H": H, "state": state}
    if st["case"]["train"]:
        dQ, dK, dV, dstate = aa.decay_backward(st["Q"], st["K"], st["V"], st["dH"], st["log_decay"], dstate=st["dstate"], **how)
        out |= {"dQ": dQ, "dK": dK, "dV": dV}
        if dstate is not None:
            out["dstate"] = dstate
    return out


def own_step(st):
    import linear_complexity_anchor_gb300 as aa
    H = aa.decay_step(st["Q"], st["K"], st["V"], st["log_decay"], st["states"], st["slots"], scale=st["scale"])
    return {"H": H, "states": st["states"]}


def own_norm(st):
    import linear_complexity_anchor_gb300 as aa
    c = st["case"]
    if c["bits8"]:
        Y, scales, S = aa.add_norm_8bit(st["X"], st["R"], st["w"], eps=EPS, group=c["group"])
        out = {"Y": Y, "scales": scales}
    else:
        Y, S = aa.add_norm(st["X"], st["R"], st["w"], eps=EPS)
        out = {"Y": Y}
    if st["R"] is not None:
        out["S"] = S
    if c["train"]:
        out["dX"], out["dw"] = aa.add_norm_backward(S, st["dY"], st["w"], dS=st["dS"], eps=EPS)
    return out


def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return own_norm(state) if own else plain_norm(state)
    if op == "step":
        return own_step(state) if own else plain_step(state)
    return own_decay(state) if own else plain_decay(state)


# ---------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        x = c["rows"] * c["D"]
        # X in; R in and the sum out; Y out; in training dY and dS in, dX out
        moved = x * size * (3 if c["residual"] else 1) + x * (1 if c["bits8"] else size) + (3 * x * size if c["train"] else 0)
        if c["bits8"]:
            moved += c["rows"] * 4 * (-(-c["D"] // (c["group"] or c["D"])))
        return {"bytes": moved, "flops": x * (16 if c["train"] else 7)}
    x, s = c["B"] * c["heads"] * c["n"] * c["d"], c["B"] * c["heads"] * c["d"] * c["d"]
    # a token's k v^T to the state, and q times the state: 4 d^2
    if c["op"] == "step":
        return {"bytes": 4 * x * size + 2 * s * 4, "flops": 4 * x * c["d"]}
    share = 0.625 if c["ragged"] else 1.0  # the mean length over n
    states = (4 if c["train"] else 2) if c["state"] else 1
    # Q, K, V in, H out; in training dH in, dQ, dK, dV out, and five products where the forward has two
    moved = x * size * ((4 * share + 4) if c["train"] else (3 * share + 1)) + states * s * 4
    return {"bytes": moved, "flops": x * share * c["d"] * (14 if c["train"] else 4)}


# ---------------------------------------------------------------------- in 64 bits, from the definitions

def exact_decay(st, lengths, state):
    """Token by token: S_t = decay S_(t-1) + k_t v_t^T, h_t = scale q_t S_t; the gradients by the states backward."""
    c = st["case"]
    B, heads, n, d = st["Q"].shape
    q, k, v = (st[x].double() for x in "QKV")
    gamma = st["log_decay"].double().exp()[None, :, None, None]
    S = torch.zeros(B, heads, d, d, dtype=torch.float64, device=q.device) if state is None else state.double().clone()
    H, dQ, dK, dV = (torch.zeros(B, heads, n, d, dtype=torch.float64, device=q.device) for _ in range(4))
    train = c.get("train", False)
    dh = st["dH"].double() if train else None
    live = [torch.ones(B, 1, 1, 1, dtype=torch.bool, device=q.device)] * n if lengths is None else list(
        (torch.arange(n, device=q.device)[:, None] < lengths[None, :])[:, :, None, None, None])
    for t in range(n):
        S = torch.where(live[t], S * gamma + k[:, :, t, :, None] * v[:, :, t, None, :], S)
        H[:, :, t] = st["scale"] * (q[:, :, t, None, :] @ S)[:, :, 0] * live[t][..., 0]
        if train:
            dQ[:, :, t] = st["scale"] * (S @ dh[:, :, t, :, None])[..., 0] * live[t][..., 0]
    out = {"H": H, "state": S}
    if train:
        G = torch.zeros_like(S) if st["dstate"] is None else st["dstate"].double().clone()
        for t in reversed(range(n)):
            G = torch.where(live[t], G + st["scale"] * q[:, :, t, :, None] * dh[:, :, t, None, :], G)
            dK[:, :, t] = (G @ v[:, :, t, :, None])[..., 0] * live[t][..., 0]
            dV[:, :, t] = (k[:, :, t, None, :] @ G)[:, :, 0] * live[t][..., 0]
            G = torch.where(live[t], G * gamma, G)
        out |= {"dQ": dQ, "dK": dK, "dV": dV}
        if st["state"] is not None:
            out["dstate"] = G
    return out


def exact_step(st):
    slots = torch.arange(st["case"]["B"], device=st["Q"].device) if st["slots"] is None else st["slots"].long()
    got = exact_decay(st, None, st["states"][slots])
    states = st["states"].double()
    states[slots] = got["state"]
    return {"H": got["H"], "states": states}


def exact_norm(st):
    c = st["case"]
    s = st["X"].double()
    out = {}
    if st["R"] is not None:
        out["S"] = s + st["R"].double()
        s = out["S"].to(st["X"].dtype).double()  # the norm is that of the sum as it is kept
    w, size = st["w"].double(), ((s * s).sum(-1, keepdim=True) / c["D"] + EPS).sqrt()
    y = s / size * w
    if c["bits8"]:
        each = c["group"] or c["D"]
        parts = y.split(each, -1)
        scales = torch.stack([p.abs().max(-1).values / TOP for p in parts], -1)
        over = torch.where(scales == 0, 1.0, scales).repeat_interleave(each, -1)[:, : c["D"]]
        return out | {"Y": y / over, "scales": scales}
    out["Y"] = y
    if c["train"]:
        dy = st["dY"].double()
        out["dw"] = (dy * s / size).sum(0)
        a = dy * w / size
        out["dX"] = a - s * (a * s).sum(-1, keepdim=True) / (c["D"] * size * size) + st["dS"].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(st)
    return exact_step(st) if case["op"] == "step" else exact_decay(st, st["lengths"], st["state"])
