"""GPU: the operators of a layer with decaying states one after the other, as a model uses them, in training and in serving;
places in memory past 32 bits; calls on two streams at once."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.decay_reference import add_norm_reference, decay_reference
from tests.ops_reference import assert_within

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def weights(heads, d, D, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return {"norm": (1 + 0.1 * n(D)).to(dtype), "qkv": (n(3 * heads * d, D) * D ** -0.5).to(dtype), "out": (n(D, heads * d) * (heads * d) ** -0.5).to(dtype),
            "log_decay": -torch.exp2(-2.0 - torch.arange(heads, device="cuda").float())}


def projected(y, w, heads, d):
    B, n, _ = y.shape
    return (y @ w["qkv"].to(y.dtype).T).reshape(B, n, 3, heads, d).permute(2, 0, 3, 1, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step(aa, dtype):
    """Residual, norm, projections, attention, and back through all of them, against autograd in 64 bits."""
    B, n, heads, d, D = 2, 150, 3, 64, 192
    w = weights(heads, d, D, DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(3)
    X, R, dO, dS = (torch.randn(B, n, D, generator=g, device="cuda").to(DT[dtype]) for _ in range(4))
    L = torch.tensor([n, 70], dtype=torch.int32, device="cuda")

    Y, S = aa.add_norm(X, R, w["norm"])
    q, k, v = projected(Y, w, heads, d)
    H = aa.decay_forward(q, k, v, w["log_decay"], L)
    O = H.transpose(1, 2).reshape(B, n, heads * d) @ w["out"].T
    dH = (dO @ w["out"]).reshape(B, n, heads, d).transpose(1, 2)
    dq, dk, dv, none = aa.decay_backward(q, k, v, dH, w["log_decay"], L)
    assert none is None
    dqkv = torch.stack((dq, dk, dv)).permute(1, 3, 0, 2, 4).reshape(B, n, -1)
    dX, dw = aa.add_norm_backward(S, dqkv @ w["qkv"], w["norm"], dS=dS)

    x = {name: t.double().requires_grad_() for name, t in (("X", X), ("R", R), ("norm", w["norm"]))}
    s = x["X"] + x["R"]
    y = s / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt() * x["norm"]
    q, k, v = projected(y, {"qkv": w["qkv"].double()}, heads, d)
    i = torch.arange(n, device="cuda")
    on = (i[None] < L[:, None])[:, None, :, None]
    decay = torch.where(i[:, None] >= i[None], (w["log_decay"].double()[:, None, None] * (i[:, None] - i[None])).exp(), 0.0)
    h = ((q @ k.mT) * d ** -0.5 * decay * on.mT) @ v * on
    o = h.transpose(1, 2).reshape(B, n, heads * d) @ w["out"].double().T
    torch.autograd.backward((o, s), (dO.double(), dS.double()))
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    # eight results rounded one after the other, each by half a step at most: in the root of the mean square less
    bound = 8 * torch.finfo(DT[dtype]).eps / 2 if dtype == "bf16" else 2e-5
    for name, got, want in (("O", O, o), ("dX", dX, x["X"].grad), ("dX as dR", dX, x["R"].grad), ("dw", dw, x["norm"].grad)):
        assert rel(got, want.detach()) <= bound, name


def test_serving(aa):
    """A batch of prompts, then tokens one by one over a pool of states, with 8-bit norms before the projections: the same as all
    tokens at once."""
    B, n, heads, d, D = 3, 200, 4, 64, 256
    w = weights(heads, d, D, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(5)
    X, R = (torch.randn(B, n + 8, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    L = torch.tensor([200, 64, 131], dtype=torch.int32, device="cuda")

    def layer_input(x, r):
        Y, scales, S = aa.add_norm_8bit(x, r, w["norm"], group=128)
        ref, (y, off) = add_norm_reference(x, r, w["norm"], 1e-6)
        over = scales.double().repeat_interleave(128, -1)
        assert torch.equal(S, ref)
        assert_within(Y.double() * over, (y, 2.0 ** -4 * y.abs() + 2.0 ** -10 * over + 4 * off), "norm")
        return projected((Y.float() * over.float()).bfloat16(), w, heads, d)

    q, k, v = layer_input(X, R)
    H, states = aa.decay_forward(q[:, :, :n], k[:, :, :n], v[:, :, :n], w["log_decay"], L, return_state=True)
    pool = torch.zeros(7, heads, d, d, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = states
    seen = [[q[b:b + 1, :, :int(L[b])], k[b:b + 1, :, :int(L[b])], v[b:b + 1, :, :int(L[b])]] for b in range(B)]
    for t in range(n, n + 8):
        now = [x[:, :, t:t + 1] for x in (q, k, v)]
        h = aa.decay_step(*now, w["log_decay"], pool, slots)
        for b in range(B):
            seen[b] = [torch.cat((s, x[b:b + 1]), 2) for s, x in zip(seen[b], now)]
            ref = decay_reference(*seen[b], w["log_decay"], None, None, d ** -0.5)
            assert_within(h[b:b + 1], tuple(x[:, :, -1:] for x in ref["H"]), (t, b))
            assert_within(pool[int(slots[b])][None], ref["last"], (t, b, "state"))
    assert not pool[[1, 2, 4, 6]].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_places(aa, dtype):
    """Entries, rows and slots more than 2^31 elements apart."""
    far = (1 << 31) + 64
    buf = torch.empty(far + 2 * 300 * 64, dtype=DT[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    near = [torch.randn(2, 2, 300, 64, generator=g, device="cuda").to(DT[dtype]) for _ in range(4)]
    rate = torch.tensor([-0.01, -0.2], device="cuda")
    x = buf.as_strided((2, 2, 300, 64), (far, 300 * 64, 64, 1))
    x.copy_(near[0])
    want = aa.decay_forward(*near[:3], rate)
    assert torch.equal(aa.decay_forward(x, *near[1:3], rate), want)
    for a, b in zip(aa.decay_backward(x, *near[1:4], rate)[:3], aa.decay_backward(*near, rate)[:3]):
        assert torch.equal(a, b)
    x.zero_()
    aa.decay_forward(*near[:3], rate, H=x)
    assert torch.equal(x, want)
    rows = buf.as_strided((2, 256), (far, 1))
    rows.copy_(near[0].reshape(-1, 256)[:2])
    flat = rows.contiguous()
    for a, b in zip(aa.add_norm(rows, flat), aa.add_norm(flat, flat)):
        assert torch.equal(a, b)
    assert torch.equal(aa.add_norm_backward(rows, flat)[0], aa.add_norm_backward(flat, flat)[0])
    del x, rows, buf
    count = (1 << 31) // (2 * 64 * 64) + 2
    pool = torch.empty(count, 2, 64, 64, device="cuda")
    slots = torch.tensor([count - 1, 0], dtype=torch.int32, device="cuda")
    few = torch.randn(2, 2, 64, 64, generator=g, device="cuda")
    pool[slots.long()] = few
    one = [t[:, :, :1] for t in near[:3]]
    assert torch.equal(aa.decay_step(*one, rate, pool, slots), aa.decay_step(*one, rate, few))
    assert torch.equal(pool[slots.long()], few)


def test_two_streams(aa):
    """Calls that take workspaces, at once on two streams: each with its own."""
    g = torch.Generator(device="cuda").manual_seed(8)
    sets = [[torch.randn(1, 2, 4000, 64, generator=g, device="cuda").bfloat16() for _ in range(4)] for _ in range(2)]
    rows = [torch.randn(900, 768, generator=g, device="cuda").bfloat16() for _ in range(2)]
    rate, w = torch.tensor([-0.001, -0.03], device="cuda"), torch.ones(768, device="cuda").bfloat16()
    run = lambda i: (*aa.decay_forward(*sets[i][:3], rate, return_state=True), *aa.decay_backward(*sets[i], rate)[:3], *aa.add_norm_backward(rows[i], rows[i], w))  # noqa: E731
    want = [run(0), run(1)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [None, None]
        for i in range(2):
            with torch.cuda.stream(side[i]):
                got[i] = run(i)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_scores_of_any_size(aa):
    """Inputs up to the type's end, a scale of 0, negative and large ones: finite where the result is."""
    for dtype in DT.values():
        q, k, v = (torch.randn(1, 2, 140, 64, device="cuda").to(dtype) for _ in range(3))
        rate = torch.tensor([-0.1, -3.0], device="cuda")
        base = aa.decay_forward(q, k, v, rate, scale=1.0)
        assert not aa.decay_forward(q, k, v, rate, scale=0.0).any()
        assert torch.equal(aa.decay_forward(q, k, v, rate, scale=-1.0), -base)
        assert torch.equal(aa.decay_forward(q * 2.0 ** 60, k, v, rate, scale=2.0 ** -60), base)
        assert torch.equal(aa.decay_forward(q, k * 2.0 ** 50, v * 2.0 ** -50, rate, scale=1.0), base)
        assert math.isfinite(float(aa.decay_forward(q, k, v, rate, scale=2.0 ** 100).float().abs().max()))


def test_two_graphs_at_once(aa):
    # both take workspaces (segments, sums of a weight's gradient), and are replayed on streams of their own
    g = torch.Generator(device="cuda").manual_seed(21)
    graphs, wants, outs, runs = [], [], [], []
    for B, heads, n, d in ((1, 2, 1700, 64), (1, 3, 1500, 128)):
        Q, K, V, dH = (torch.randn(B, heads, n, d, generator=g, device="cuda").bfloat16() for _ in range(4))
        X, dY = (torch.randn(n, heads * d, generator=g, device="cuda").bfloat16() for _ in range(2))
        w = torch.rand(heads * d, generator=g, device="cuda")
        rate = -1.0 / torch.linspace(30.0, 900.0, heads, device="cuda")

        def run(Q=Q, K=K, V=V, dH=dH, X=X, dY=dY, w=w, rate=rate):
            H, last = aa.decay_forward(Q, K, V, rate, return_state=True)
            return (H, last, *aa.decay_backward(Q, K, V, dH, rate)[:3], *aa.add_norm_backward(X, dY, w))

        runs.append(run)  # (with its inputs, which the graphs read)
        wants.append([t.clone() for t in run()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for out in outs:
            for t in out:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for out, want in zip(outs, wants):
            assert all(torch.equal(a, b) for a, b in zip(out, want))
