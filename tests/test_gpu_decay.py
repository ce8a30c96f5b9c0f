"""GPU: attention with decaying states, forward, backward and token by token, against its definition in 64 bits with bounds
that count the kernels' roundings (tests/decay_reference.py)."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.decay_reference import decay_reference, lengths_of, powers
from tests.ops_reference import assert_within, half_step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def make(seed, B, heads, n, d, dtype, tokens=False, state=False, ragged=False, train=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows():
        x = torch.randn((B, n, heads, d) if tokens else (B, heads, n, d), generator=g, device="cuda").to(DT[dtype])
        return x.transpose(1, 2) if tokens else x

    x = {name: rows() for name in ("Q", "K", "V")}
    # from a head that keeps its token alone to one that loses nothing
    some = torch.tensor([-0.02, -0.0005, -0.3, 0.0, -4.0, -math.inf, -1e-5, 0.7], device="cuda")
    x["log_decay"] = some[torch.arange(heads, device="cuda") % 8].contiguous()
    x["lengths"] = None
    if ragged:
        L = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        L[0] = 0 if seed % 2 else n
        if B > 2:
            L[1], L[2] = n + 5, -3
        x["lengths"] = L
    x["state"] = torch.randn(B, heads, d, d, generator=g, device="cuda") * 3 if state else None
    if train:
        x["dH"] = rows()
        x["dlast"] = torch.randn(B, heads, d, d, generator=g, device="cuda") if state else None
    return x


def forward(aa, x, **how):
    return aa.decay_forward(x["Q"], x["K"], x["V"], x["log_decay"], x["lengths"], state=x["state"], return_state=True, **how)


def backward(aa, x, **how):
    return aa.decay_backward(x["Q"], x["K"], x["V"], x["dH"], x["log_decay"], x["lengths"], state=x["state"], dstate=x["dlast"], **how)


def check(aa, x, scale, what, train=False):
    ref = decay_reference(x["Q"], x["K"], x["V"], x["log_decay"], x["lengths"], x["state"], scale, x.get("dH"), x.get("dlast"))
    H, last = forward(aa, x, scale=scale)
    got = {"H": H, "last": last}
    if train:
        got |= dict(zip(("dQ", "dK", "dV", "dstate"), backward(aa, x, scale=scale)))
    for name, t in got.items():
        if t is None:
            assert name == "dstate" and x["state"] is None
            continue
        assert_within(t, ref[name], f"{what}: {name}")
        if name in ("H", "dQ", "dK", "dV"):
            assert t.dtype == x["Q"].dtype and t.stride() == torch.empty_like(x["Q"]).stride()


LENGTHS = (1, 2, 8, 9, 63, 64, 65, 127, 128, 129, 200, 256, 257, 515)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_forward(aa, dtype, d):
    for i, n in enumerate(LENGTHS):
        x = make(i, 1 + i % 3, 1 + (3 * i) % 8, n, d, dtype, tokens=i % 2 == 0, state=i % 3 != 0, ragged=i % 2 == 1)
        check(aa, x, (0.3, d ** -0.5, -1.0)[i % 3], f"{dtype} d {d} n {n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_backward(aa, dtype, d):
    for i, n in enumerate(LENGTHS):
        x = make(50 + i, 1 + i % 3, 1 + (5 * i) % 8, n, d, dtype, tokens=i % 2 == 1, state=i % 3 != 1, ragged=i % 4 < 2, train=True)
        check(aa, x, (d ** -0.5, 0.4, 1.0)[i % 3], f"{dtype} d {d} n {n}", train=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,heads,n,d", [(1, 1, 4000, 64), (1, 2, 2049, 128), (2, 1, 3001, 32), (3, 2, 1100, 64), (1, 1, 2600, 16), (40, 8, 1200, 64)])
def test_long(aa, dtype, B, heads, n, d):
    """Few heads whose tokens are cut into segments; and many, which are not."""
    for state, ragged in ((True, True), (False, False)):
        x = make(7, B, heads, n, d, dtype, state=state, ragged=ragged, train=True)
        if not ragged:
            x["log_decay"] = torch.linspace(-0.01, -0.0001, heads, device="cuda")
        check(aa, x, d ** -0.5, f"{dtype} {B} x {heads} x {n} x {d} state {state}", train=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rounding(aa, dtype, d):
    """The results as a whole are off by little more than a rounding of each kind: 1.5 times a lone rounding of the result
    (0.6 of half a step in the root of the mean square), the states by fp32's."""
    x = make(3, 2, 4, 1500, d, dtype, state=True, train=True)
    x["log_decay"] = torch.tensor([-0.03, -0.004, -0.0005, -0.0001], device="cuda")
    ref = decay_reference(x["Q"], x["K"], x["V"], x["log_decay"], None, x["state"], d ** -0.5, x["dH"], x["dlast"])
    H, last = forward(aa, x)
    dQ, dK, dV, dstate = backward(aa, x)
    rel = lambda t, name: float((t.double() - ref[name][0]).norm() / ref[name][0].norm())  # noqa: E731
    for name, t in (("H", H), ("dQ", dQ), ("dK", dK), ("dV", dV)):
        assert rel(t, name) <= (1.5 * 0.6 * half_step(t.dtype) * (1 if dtype == "bf16" else 40)), name
    for name, t in (("last", last), ("dstate", dstate)):
        assert rel(t, name) <= 1e-5, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [1, 160], ids=["segments", "whole"])
def test_a_state_that_loses_nothing(aa, dtype, heads):
    # Positive numbers whose sum is longer than 2^8 chunks: a sum that is cut off, not rounded, loses half a step of itself at each
    # addition.  One rounding to nearest a chunk (of 64 rows at least: 2^-24 each), and the sum of a chunk, of 16 products
    # at a time, each of which may lose as many last bits (8 products of 2^-20 x 2^-1 at most).
    n, d = 32768, 64
    g = torch.Generator(device="cuda").manual_seed(heads)
    K, V = ((torch.rand(1, 1, n, d, generator=g, device="cuda") + 0.5).to(DT[dtype]).expand(1, heads, n, d).contiguous() for _ in range(2))
    last = aa.decay_forward(K, K, V, torch.zeros(heads, device="cuda"), None, return_state=True)[1]
    want = K[0, 0].double().t() @ V[0, 0].double()
    off = ((last.double() - want) / want).abs().max().item()
    assert off < (n // 64) * 2.0 ** -24 + 8 * 2.0 ** -21, off
    # bf16 rows count as they are (weights of 1): chunks of 128
    if dtype == "bf16":
        assert off < (n // 128) * 2.0 ** -24 + 8 * 2.0 ** -21, off


@pytest.mark.parametrize("dtype,B,n", [("bf16", 8, 65536), ("f32", 8, 32768), ("f32", 1, 32768), ("bf16", 1, 4096), ("f32", 1, 4096)],
                         ids=["bf16", "f32", "segments", "steps-bf16", "steps-f32"])
def test_a_state_that_fades_slowly(aa, dtype, B, n):
    # Tokens of zeros: the state behind them is exp(n log_decay) of the one before.  A factor that is rounded the same way each time
    # would add up to n / 64 2^-25 of it (token by token: n 2^-25).  What may be left: one rounding to nearest for each
    # factor, of 2^-24 / sqrt(12) in the mean, and what is made good every 32 factors only.
    heads, d = 32, 64
    steps = n == 4096
    g = torch.Generator(device="cuda").manual_seed(n + B)
    zero = torch.zeros(B, heads, n, d, device="cuda", dtype=DT[dtype])
    rate = -1.0 / torch.linspace(2000 if steps else n, 6000 if steps else 4 * n, heads, device="cuda")
    X = torch.randn(B, heads, d, d, generator=g, device="cuda")
    if steps:
        last = X.clone()
        aa.decay_step(zero, zero, zero, rate, last)
    else:
        last = aa.decay_forward(zero, zero, zero, rate, None, state=X, return_state=True)[1]
    want = X.double() * torch.exp(rate.double() * n).view(1, heads, 1, 1)
    off = ((last - want).square().sum((0, 2, 3)) / want.square().sum((0, 2, 3))).sqrt()
    factors = n if steps else n // 64
    bound = 2 * (factors * 2.0 ** -48 / 12) ** 0.5 + (2.0 ** -24 if steps else 32 * 2.0 ** -25)
    assert off.max().item() < 2 * bound, (off.max().item(), bound)


@pytest.mark.parametrize("B,heads,n,d", [(4, 8, 197, 64), (2, 8, 3000, 64), (1, 8, 9000, 128), (40, 8, 1000, 32), (20, 8, 700, 128)])
def test_states_are_fp32_results(aa, B, heads, n, d):
    # What the rows of bf16 leave is less than 2^-18 in the mean where the decay leaves e^-2 of it, 2^-24 elsewhere; the sum of a
    # chunk is cut off at each of 8 products (2^-25 in the mean), and one rounding a chunk is to nearest: 0.8e-6 in all.
    x = make(d + n, B, heads, n, d, "bf16", state=True, train=True, ragged=True)
    x["log_decay"] = -1.0 / torch.tensor([3.0, 30.0, 60.0, 130.0, 400.0, 900.0, 4000.0, 1e6], device="cuda")
    last, first = forward(aa, x, scale=0.5)[1], backward(aa, x, scale=0.5)[3]
    L, i = lengths_of(x["lengths"], B, n, "cuda"), torch.arange(n, device="cuda")
    on = (i[None] < L[:, None])[:, None, :, None]
    q, k, v, dh = (torch.where(on, x[name].double(), 0.0) for name in ("Q", "K", "V", "dH"))
    whole = powers(x["log_decay"], L).transpose(0, 1)[..., None, None]
    rest = powers(x["log_decay"], L[:, None] - 1 - i[None]).transpose(0, 1)[..., None]
    ahead = powers(x["log_decay"], i + 1)[None, ..., None]
    for got, want in ((last, (k * rest).mT @ v + whole * x["state"].double()), (first, 0.5 * (q * ahead).mT @ dh + whole * x["dlast"].double())):
        off = ((got.double() - want).square().sum((0, 2, 3)) / want.square().sum((0, 2, 3))).sqrt()
        assert off.max().item() < 1e-6, off


@pytest.mark.parametrize("rate", [0.0, -0.0, 0.7, -1e-30], ids=["zero", "minus-zero", "above", "tiny"])
@pytest.mark.parametrize("B,n", [(1, 2000), (30, 500)])
def test_states_of_heads_that_lose_nothing_are_fp32_results(aa, B, n, rate):
    # as above, with weights that are a scale alone, which is no bf16 number
    x = make(n, B, 6, n, 64, "bf16", state=True, train=True)
    x["log_decay"] = torch.full((6,), rate, device="cuda")
    first = backward(aa, x, scale=0.3)[3].double()
    want = 0.3 * x["Q"].double().mT @ x["dH"].double() + x["dlast"].double()
    assert ((first - want).square().sum() / want.square().sum()).sqrt().item() < 1e-6


@pytest.mark.parametrize("d", [16, 64, 128])
def test_gradients_by_differences(aa, d):
    """H and the last states are linear in each of Q, K, V and the first states, so that a difference of any size is the
    gradient's product with it."""
    x = make(11, 2, 3, 150, d, "f32", state=True, ragged=True, train=True)
    loss = lambda y: sum(float((a.double() * b.double()).sum()) for a, b in zip(forward(aa, y), (x["dH"], x["dlast"])))  # noqa: E731
    grads = dict(zip(("Q", "K", "V", "state"), backward(aa, x)))
    base = loss(x)
    g = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in grads.items():
        step = torch.randn(x[name].shape, generator=g, device="cuda")
        want = loss({**x, name: x[name] + step}) - base
        got = float((grad.double() * step.double()).sum())
        size = float(grad.double().norm() * step.double().norm())
        assert abs(got - want) <= 1e-5 * (size + abs(base)), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_behind_the_length_do_not_matter(aa, dtype):
    for n, d, B in ((200, 64, 3), (140, 128, 3), (1500, 32, 1), (5, 64, 3)):
        x = make(2, B, 2, n, d, dtype, state=True, ragged=True, train=True)
        x["lengths"] = torch.tensor([n // 3, 0, n - 1][:B], dtype=torch.int32, device="cuda")
        want = (*forward(aa, x), *backward(aa, x))
        off = (torch.arange(n, device="cuda")[None] >= x["lengths"][:, None])[:, None, :, None]
        for bad in (math.nan, math.inf):
            y = {**x, **{name: x[name].masked_fill(off, bad) for name in ("Q", "K", "V", "dH")}}
            for a, b in zip((*forward(aa, y), *backward(aa, y)), want):
                assert torch.equal(a, b)
        for t in (want[0], *want[2:5]):
            assert not t.masked_select(off.expand_as(t)).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_carry_a_sequence_on(aa, dtype):
    """Parts one after the other, each with the state behind the one before, are the whole; the last of them by tokens."""
    x = make(4, 2, 3, 400, 64, dtype, state=True)
    H, last = forward(aa, x)
    ref = decay_reference(x["Q"], x["K"], x["V"], x["log_decay"], None, x["state"], 0.125)
    state, parts = x["state"], []
    for a, b in ((0, 130), (130, 131), (131, 391)):
        h, state = aa.decay_forward(*(x[k][:, :, a:b] for k in "QKV"), x["log_decay"], state=state, return_state=True)
        parts.append(h)
    pool = torch.full((5, 3, 64, 64), 7.0, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(391, 400):
        parts.append(aa.decay_step(*(x[k][:, :, t:t + 1] for k in "QKV"), x["log_decay"], pool, slots))
    assert_within(torch.cat(parts, 2), ref["H"], "H")
    assert_within(pool[slots.long()], ref["last"], "last")
    assert bool((pool[[0, 2, 4]] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,heads,n,d", [(1, 1, 1, 16), (3, 5, 1, 32), (2, 12, 1, 64), (70, 8, 1, 64), (50, 8, 1, 128), (3, 2, 4, 128), (5, 3, 9, 64),
                                         (300, 1, 2, 16)])
def test_step(aa, dtype, B, heads, n, d):
    x = make(B, B, heads, n, d, dtype, tokens=B % 2 == 0)
    g = torch.Generator(device="cuda").manual_seed(1)
    for pooled in (False, True):
        states = torch.randn(B + 3, heads, d, d, generator=g, device="cuda")
        slots = torch.randperm(B + 3, generator=g, device="cuda")[:B].int() if pooled else None
        at = slots.long() if pooled else torch.arange(B, device="cuda")
        if pooled:  # one without a state, one past the last
            slots[0] = -1
            if B > 2:
                slots[2] = B + 3
        before = states.clone()
        ref = decay_reference(x["Q"], x["K"], x["V"], x["log_decay"], None, before[at], 0.2)
        H = aa.decay_step(x["Q"], x["K"], x["V"], x["log_decay"], states, slots, scale=0.2)
        live = torch.ones(B, dtype=torch.bool, device="cuda") if slots is None else (slots >= 0) & (slots < B + 3)
        assert_within(H[live], tuple(t[live] for t in ref["H"]), "H")
        assert not H[~live].any()
        assert_within(states[at[live]], tuple(t[live] for t in ref["last"]), "states")
        rest = torch.ones(B + 3, dtype=torch.bool, device="cuda")
        rest[at[live]] = False
        assert torch.equal(states[rest], before[rest])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_with_shared_slots(aa, dtype):
    """Requests with one slot are taken in order, as if their tokens followed one another."""
    B, heads, d = 300, 2, 64
    x = make(9, B, heads, 1, d, dtype)
    slots = torch.arange(B, dtype=torch.int32, device="cuda") % 7
    states = torch.randn(8, heads, d, d, device="cuda")
    want_states, want = states.clone(), torch.empty_like(x["Q"])
    for b in range(B):
        s = slice(b, b + 1)
        want[s] = aa.decay_step(x["Q"][s], x["K"][s], x["V"][s], x["log_decay"], want_states, slots[s])
    H = aa.decay_step(x["Q"], x["K"], x["V"], x["log_decay"], states, slots)
    assert torch.equal(H, want) and torch.equal(states, want_states)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_rows_and_given_outputs(aa, dtype):
    """Key heads shared by an expanded axis, H given as a part of a wider buffer, no tokens, no heads."""
    x = make(6, 2, 4, 90, 64, dtype, train=True)
    K1 = x["K"][:, :1]
    y = {**x, "K": K1.expand(-1, 4, -1, -1)}
    z = {**x, "K": K1.repeat(1, 4, 1, 1)}
    for a, b in zip((*forward(aa, y), *backward(aa, y)), (*forward(aa, z), *backward(aa, z))):
        assert a is b is None or torch.equal(a, b)
    wide = torch.full((2, 4, 92, 128), 5.0, device="cuda", dtype=DT[dtype])
    H, _ = forward(aa, z, H=wide[:, :, 1:91, 64:])
    assert H.data_ptr() == wide[:, :, 1:91, 64:].data_ptr() and torch.equal(H, forward(aa, z)[0])
    assert bool((wide[..., :64] == 5).all()) and bool((wide[:, :, 0] == 5).all()) and bool((wide[:, :, 91] == 5).all())
    none = {**make(1, 2, 3, 0, 64, dtype, state=True), "dH": x["dH"][:, :3, :0], "dlast": torch.ones(2, 3, 64, 64, device="cuda")}
    H, last = forward(aa, none)
    assert H.shape == (2, 3, 0, 64) and torch.equal(last, none["state"])
    assert torch.equal(backward(aa, none)[3], none["dlast"])
    assert not forward(aa, {**none, "state": None})[1].any()
    assert aa.decay_forward(*(x[k][:, :0] for k in "QKV"), x["log_decay"][:0]).shape == (2, 0, 90, 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_on_a_stream_and_in_a_graph(aa, dtype):
    x = make(8, 1, 2, 1300, 64, dtype, state=True, ragged=True, train=True)
    s = make(8, 4, 3, 1, 64, dtype)
    first = torch.randn(4, 3, 64, 64, device="cuda")
    states = first.clone()

    def run():
        return (*forward(aa, x), *backward(aa, x), aa.decay_step(s["Q"], s["K"], s["V"], s["log_decay"], states))

    want = [t.clone() for t in run()] + [states.clone()]
    states.copy_(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [t.clone() for t in run()] + [states.clone()]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        states.copy_(first)
        for t in out:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([*out, states], want))
