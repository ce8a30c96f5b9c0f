"""GPU: cross attention, forward and backward, against its definition in 64 bits, with bounds that count the kernels'
roundings (tests/ops_reference.py); layouts, lengths, streams, captured graphs and what the results may not depend on."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.ops_reference import assert_within, cross_reference

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def make(seed, B, heads, kv, n, s, d, dtype, tokens=False, gain=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def one(h, rows, by=1.0):
        shape = (B, rows, h, d) if tokens else (B, h, rows, d)
        x = (by * torch.randn(shape, generator=g, device="cuda")).to(DT[dtype])
        return x.transpose(1, 2) if tokens else x

    return one(heads, n, gain), one(kv, s), one(kv, s), one(heads, n)


def lengths_of(kind, B, s):
    """none; the whole range with empty and full entries in turn; or a number for all."""
    if kind is None:
        return None
    if kind == "mixed":
        some = [0, s, 1, s // 2, max(0, s - 1), min(s, 64), min(s, 65), min(s, 128), min(s, 129)]
        return torch.tensor([some[i % len(some)] for i in range(B)], dtype=torch.int32, device="cuda")
    return torch.full((B,), kind, dtype=torch.int32, device="cuda")


def check(aa, seed, B, heads, kv, n, s, d, dtype, lengths=None, tokens=False, train=True, scale=None):
    Q, K, V, dH = make(seed, B, heads, kv, n, s, d, dtype, tokens)
    L = lengths_of(lengths, B, s)
    c = d ** -0.5 if scale is None else scale
    H, lse = aa.cross_forward(Q, K, V, L, scale=scale, return_lse=True)
    ref = cross_reference(Q, K, V, L, c, dH if train else None)
    what = f"{dtype} B{B} heads{heads}/{kv} n{n} s{s} d{d} {lengths}"
    assert_within(H, ref["H"], "H " + what)
    assert_within(lse, ref["lse"], "lse " + what)
    if train:
        for name, got in zip(("dQ", "dK", "dV"), aa.cross_backward(Q, K, V, H, lse, dH, L, scale=scale)):
            assert_within(got, ref[name], name + " " + what)
    return Q, K, V, dH, L, H, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("shape", [(2, 2, 2, 1, 1), (1, 1, 1, 3, 2), (2, 3, 1, 17, 63), (9, 2, 2, 65, 200), (1, 4, 2, 130, 129),
                                   (2, 2, 1, 300, 515)])
def test_shapes(aa, dtype, d, shape):
    check(aa, sum(shape) + d, *shape, d, dtype, lengths="mixed" if shape[0] > 1 else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,lengths", [((9, 4, 2, 1, 700, 64), "mixed"), ((1, 12, 12, 1, 1500, 64), None), ((1, 1, 1, 1, 9000, 128), None),
                                           ((3, 8, 1, 1, 2050, 128), "mixed"), ((2, 8, 2, 5, 1300, 32), "mixed"), ((1, 32, 1, 4, 640, 128), None),
                                           ((2, 64, 2, 1, 333, 16), "mixed"), ((4, 2, 2, 2, 5000, 64), 0),
                                           ((20, 16, 8, 1, 8200, 128), "mixed"), ((20, 8, 8, 3, 16400, 64), None)])
def test_few_queries(aa, dtype, shape, lengths):
    check(aa, 7, *shape, dtype, lengths=lengths, train=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_few_queries_of_many_entries(aa, dtype, d):
    """A token of so many entries that no key axis is cut; what is summed last counts, and every time the same."""
    Q, K, V, _, L, H, _ = check(aa, 17, 40, 16, 8, 1, 2900, d, dtype, lengths="mixed", train=False)
    for _ in range(20):
        assert torch.equal(H, aa.cross_forward(Q, K, V, L))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("s", [1, 16, 31, 77, 112, 127, 128])
def test_short_states(aa, dtype, d, s):
    """All states in one tile: rows of several tiles, of shared heads, and single ones."""
    check(aa, s, 9, 4, 2, 197, s, d, dtype, lengths="mixed", train=s == 77)
    check(aa, s, 9, 8, 2, 1, s, d, dtype, lengths="mixed", train=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_tiles(aa, dtype):
    """More row tiles and key tiles than any stage or part, with heads that share keys."""
    check(aa, 3, 2, 4, 2, 1030, 1100, 64, dtype, lengths="mixed")
    check(aa, 4, 1, 2, 1, 700, 1290, 128, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(aa, dtype, scale):
    check(aa, 5, 2, 2, 2, 70, 150, 64, dtype, lengths="mixed", scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_scores(aa, dtype):
    """Keys whose scores grow tile by tile: the running maximum moves at every tile."""
    B, heads, n, s, d = 1, 2, 200, 900, 64
    Q, K, V, dH = make(11, B, heads, heads, n, s, d, dtype)
    K = (K.float() + Q.float().mean(2, keepdim=True).sign() * (torch.arange(s, device="cuda")[None, None, :, None] / s * 3)).to(K.dtype)
    Q = (Q.float() * 0.5 + Q.float().mean(2, keepdim=True).sign()).to(Q.dtype)
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    ref = cross_reference(Q, K, V, None, d ** -0.5, dH)
    assert_within(H, ref["H"], "H")
    assert_within(lse, ref["lse"], "lse")
    for name, got in zip(("dQ", "dK", "dV"), aa.cross_backward(Q, K, V, H, lse, dH)):
        assert_within(got, ref[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 2, 150, 300, 64), (2, 4, 2, 300, 260, 128), (2, 8, 1, 1, 700, 128), (3, 2, 2, 40, 100, 64), (40, 8, 4, 1, 900, 128)])
def test_huge_scores(aa, dtype, shape):
    """Scores of tens of thousands: one state takes a row's whole weight, and exponents differ by more than fp32 has."""
    Q, K, V, _ = make(31, *shape, dtype)
    Q, K = Q * 300, K * 30
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    x = (Q.double() @ K.double().repeat_interleave(shape[1] // shape[2], 1).mT) * shape[5] ** -0.5
    assert float(x.abs().max()) > 1.5e4 and bool(H.isfinite().all())
    # scores are off by d roundings of fp32 of their products at the most: rows whose best state is ahead by more than that
    two = x.topk(2, -1)
    off = (shape[5] + 20) * 2.0 ** -23 * (Q.double().abs() @ K.double().abs().repeat_interleave(shape[1] // shape[2], 1).mT).amax(-1) * shape[5] ** -0.5
    sure = two.values[..., 0] - two.values[..., 1] > 40 + 2 * off
    assert float(sure.double().mean()) > 0.5
    best = V.repeat_interleave(shape[1] // shape[2], 1).gather(2, two.indices[..., :1].expand(*H.shape))
    # H = p v / p for one weight p: p is 2 to the rounding of c times the maximum, 2^(2^-24 c x) and not 1, and is
    # rounded once (bf16: half a step u) before it meets v; the product, the quotient and H are rounded once each
    assert bool(((H - best).double().abs()[sure] <= (2 + 2.0 ** -6) * torch.finfo(DT[dtype]).eps / 2 * best.double().abs()[sure]
                 * (1 if dtype == "bf16" else 2)).all())
    assert bool(((lse.double() - two.values[..., 0]).abs()[sure] <= off[sure] + 2.0 ** -20 * two.values[..., 0].abs()[sure]).all())


def test_offsets_past_32_bits(aa):
    """Batch entries, heads and rows further apart than 2^32 bytes, and 2^31 elements, of one buffer."""
    buf = torch.zeros(3 * 2 ** 31, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    # (the last: whether parts of one buffer can be told apart, which the heads' stride decides)
    for shape, strides, inside in (((2, 2, 70, 64), (2 ** 32, 2 ** 12, 2 ** 14, 1), True), ((2, 2, 130, 64), (2 ** 12, 2 ** 32, 2 ** 13, 1), False),
                                   ((1, 2, 140, 64), (64, 2 ** 12, 2 ** 25, 1), True)):
        views = [buf.as_strided(shape, strides, i * 2 ** 10) for i in range(3)]
        for v in views:
            v.copy_(torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16))
        Q, K, V = (v.contiguous() for v in views)
        H, lse = aa.cross_forward(*views, return_lse=True)
        assert torch.equal(H, aa.cross_forward(Q, K, V))
        out = buf.as_strided(shape, strides, 3 * 2 ** 10) if inside else torch.empty_like(H)
        aa.cross_forward(*views, H=out)
        assert torch.equal(out, H)
        dH = Q * 0.5
        for a, b in zip(aa.cross_backward(*views, out, lse, dH), aa.cross_backward(Q, K, V, H, lse, dH)):
            assert torch.equal(a, b)
        table = aa.rope_table(64)
        assert torch.equal(aa.rope(views[0], table), aa.rope(Q, table))
        want = aa.norm_rope(Q, K, table)
        got = aa.norm_rope(views[0], views[1], table, out=(out, None))
        assert torch.equal(out, want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 128])
def test_strides(aa, dtype, d):
    """Token-major projections, and parts of one buffer; results in the same order of axes, or dense."""
    check(aa, 8, 3, 4, 2, 100, 140, d, dtype, lengths="mixed", tokens=True)
    B, heads, n, s = 2, 3, 90, 150
    g = torch.Generator(device="cuda").manual_seed(1)
    both = torch.randn((B, s, 2, heads, d), generator=g, device="cuda").to(DT[dtype])
    K, V = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    Q = torch.randn((B, n, heads, 2 * d), generator=g, device="cuda").to(DT[dtype])[..., :d].transpose(1, 2)
    dH = torch.randn((B, heads, n, d), generator=g, device="cuda").to(DT[dtype])
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    ref = cross_reference(Q, K, V, None, d ** -0.5, dH)
    assert_within(H, ref["H"], "H")
    for name, got in zip(("dQ", "dK", "dV"), aa.cross_backward(Q, K, V, H, lse, dH)):
        assert_within(got, ref[name], name)
    out = torch.full((B, n, heads, d), 7.0, device="cuda", dtype=DT[dtype])
    assert aa.cross_forward(Q, K, V, H=out.transpose(1, 2)).data_ptr() == out.data_ptr()
    assert torch.equal(out.transpose(1, 2), H)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_shared_by_the_batch(aa, dtype):
    """K and V expanded over the batch (and over heads): gradients for each entry, their sum the shared one's."""
    B, heads, n, s, d = 3, 4, 150, 200, 64
    Q, _, _, dH = make(2, B, heads, heads, n, s, d, dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((1, 1, s, d), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    K, V = k.expand(B, heads, s, d), v.expand(B, heads, s, d)
    L = lengths_of("mixed", B, s)
    H, lse = aa.cross_forward(Q, K, V, L, return_lse=True)
    ref = cross_reference(Q, K, V, L, d ** -0.5, dH)
    assert_within(H, ref["H"], "H")
    for name, got in zip(("dQ", "dK", "dV"), aa.cross_backward(Q, K, V, H, lse, dH, L)):
        assert got.shape == ref[name][0].shape
        assert_within(got, ref[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 200])
def test_masked_states_are_not_used(aa, dtype, n):
    """Infinities and NaN behind an entry's length leave no trace; lengths out of [0, s] are taken into it."""
    B, heads, s, d = 6, 2, 300, 64
    Q, K, V, dH = make(6, B, heads, heads, n, s, d, dtype)
    L = torch.tensor([0, 1, 100, 128, 255, 300], dtype=torch.int32, device="cuda")
    H, lse = aa.cross_forward(Q, K, V, L, return_lse=True)
    grads = aa.cross_backward(Q, K, V, H, lse, dH, L)
    K2, V2 = K.clone(), V.clone()
    for b, length in enumerate(L.tolist()):
        K2[b, :, length:] = torch.tensor([math.inf, -math.inf, math.nan, torch.finfo(K.dtype).min], device="cuda").to(K.dtype).repeat(d // 4)
        V2[b, :, length:] = math.nan
    H2, lse2 = aa.cross_forward(Q, K2, V2, L, return_lse=True)
    assert torch.equal(H, H2) and torch.equal(lse, lse2)
    for a, b in zip(grads, aa.cross_backward(Q, K2, V2, H2, lse2, dH, L)):
        assert torch.equal(a, b)
    assert bool((H[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool((grads[0][0] == 0).all())
    for b, length in enumerate(L.tolist()):
        assert bool((grads[1][b, :, length:] == 0).all()) and bool((grads[2][b, :, length:] == 0).all())
    wild = torch.tensor([-5, 1, 100, 128, 255, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    assert torch.equal(H, aa.cross_forward(Q, K, V, wild))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bad_query_stays_in_its_row(aa, dtype):
    """NaN and infinities in one query row change no other row."""
    Q, K, V, _ = make(9, 2, 2, 1, 150, 200, 64, dtype)
    H = aa.cross_forward(Q, K, V)
    Q2 = Q.clone()
    Q2[0, 1, 77] = math.nan
    Q2[1, 0, 0] = math.inf
    H2 = aa.cross_forward(Q2, K, V)
    keep = torch.ones(H.shape[:3], dtype=torch.bool, device="cuda")
    keep[0, 1, 77] = keep[1, 0, 0] = False
    assert torch.equal(H[keep], H2[keep])
    assert bool(H2[0, 1, 77].isnan().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_to_do(aa, dtype):
    for B, heads, kv, n, s in ((0, 2, 2, 5, 5), (2, 2, 1, 0, 5), (2, 2, 1, 5, 0), (2, 2, 1, 0, 0)):
        Q, K, V, dH = make(1, B, heads, kv, n, s, 64, dtype)
        H, lse = aa.cross_forward(Q, K, V, return_lse=True)
        dQ, dK, dV = aa.cross_backward(Q, K, V, H, lse, dH)
        for t in (H, dQ, dK, dV):
            assert bool((t == 0).all())
        assert bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_again(aa, dtype):
    """From run to run, with other calls in between, and without lse."""
    for shape in ((2, 4, 2, 300, 700, 64), (3, 8, 2, 1, 3000, 128)):
        Q, K, V, dH = make(12, *shape, dtype)
        L = lengths_of("mixed", shape[0], shape[4])
        H, lse = aa.cross_forward(Q, K, V, L, return_lse=True)
        grads = aa.cross_backward(Q, K, V, H, lse, dH, L)
        other = make(13, 1, 2, 2, 333, 444, 64, dtype)
        for _ in range(5):
            aa.cross_forward(*other[:3])
            H2, lse2 = aa.cross_forward(Q, K, V, L, return_lse=True)
            assert torch.equal(H, H2) and torch.equal(lse, lse2) and torch.equal(H, aa.cross_forward(Q, K, V, L))
            for a, b in zip(grads, aa.cross_backward(Q, K, V, H, lse, dH, L)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first", [(2, 4, 2, 260, 600, 64), (2, 4, 2, 1100, 50, 64)])
def test_streams_and_graphs(aa, dtype, first):
    """Two calls at once on streams of their own, and two captured graphs replayed at once, give the eager bits."""
    one = make(14, *first, dtype)
    two = make(15, 4, 8, 2, 1, 2500, 64, dtype)

    def step(x, stream=None):
        Q, K, V, dH = x
        H, lse = aa.cross_forward(Q, K, V, return_lse=True, stream=stream)
        return [H, lse, *aa.cross_backward(Q, K, V, H, lse, dH, stream=stream)]

    want = [step(one), step(two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [step(x, st) for x, st in zip((one, two), streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    graphs = []
    for x, st in zip((one, two), streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = step(x)
        graphs.append((graph, out))
    for _ in range(3):
        for (graph, out), st in zip(graphs, streams):
            for t in out:
                t.fill_(5)
        torch.cuda.synchronize()
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out), a in zip(graphs, want):
            assert all(torch.equal(u, v) for u, v in zip(a, out))


def test_gradient_against_differences(aa):
    """fp32: the loss sum(H o dH) moved along a random direction, against the gradients' inner product with it."""
    Q, K, V, dH = make(21, 2, 4, 2, 9, 33, 32, "f32")
    L = torch.tensor([33, 20], dtype=torch.int32, device="cuda")
    H, lse = aa.cross_forward(Q, K, V, L, return_lse=True)
    grads = aa.cross_backward(Q, K, V, H, lse, dH, L)
    g = torch.Generator(device="cuda").manual_seed(22)
    for i, grad in enumerate(grads):
        step = torch.randn(grad.shape, generator=g, device="cuda")
        loss = []
        for e in (-1, 1):
            x = [Q, K, V]
            x[i] = x[i] + e * 2.0 ** -7 * step
            loss.append(float((aa.cross_forward(*x, L).double() * dH.double()).sum()))
        got, want = (loss[1] - loss[0]) * 2.0 ** 6, float((grad.double() * step.double()).sum())
        # the loss is off by about 300 elements' fp32 roundings (1e-6 each, random), times 2^6; the third derivative adds h^2
        assert abs(got - want) <= 5e-3 * (1 + abs(want)), (i, got, want)


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("shape,lengths", [((1, 4, 2, 1500, 50), None), ((3, 4, 1, 700, 200), "mixed"), ((2, 2, 2, 4100, 77), None),
                                           ((1, 2, 2, 40, 3000), None), ((9, 4, 2, 70, 2500), "mixed"), ((1, 1, 1, 2100, 2300), None)])
def test_backward_in_parts(aa, d, shape, lengths):
    """Few tiles that walk long: their steps are cut, and the parts' sums added by another launch, the same bits each time."""
    Q, K, V, dH, L, H, lse = check(aa, 41 + d, *shape, d, "bf16", lengths=lengths)
    first = aa.cross_backward(Q, K, V, H, lse, dH, L)
    for a, b in zip(first, aa.cross_backward(Q, K, V, H, lse, dH, L)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("s,d", [(8, 64), (64, 64), (64, 128), (384, 64), (300, 128)])
def test_few_states_lose_little(aa, s, d):
    """Up to 384 states dQ and dK are off by little more than their own rounding.  With scores near 0 all s states weigh
    alike.  H is off by its rounding and by that of the weights, together at most 1.1 * sqrt(2) of a rounding's root mean
    square e; D = dH . H by that much of dP over sqrt(s); so dQ and dK by e sqrt(1 + 2.42 / s), and by e alone where one
    tile (64 states, 128 at d = 128) has D from P and dP.  (A dS rounded once would make it e sqrt(2 + 2.42 / s).)  A tenth
    more is left for chance: they have 10^5 elements and more, 10^4 at 8 states."""
    Q, K, V, dH = make(31 + s, 4, 4, 4, 300, s, d, "bf16", gain=0.1)
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    ref = cross_reference(Q, K, V, None, d ** -0.5, dH)
    of_h = 2.42 / s if s > (64 if d <= 64 else 128) else 0.0
    for name, got in zip(("dQ", "dK"), aa.cross_backward(Q, K, V, H, lse, dH)):
        exact = ref[name][0]
        own = float((exact.to(torch.bfloat16).double() - exact).norm())
        assert float((got.double() - exact).norm()) <= 1.1 * math.sqrt(1 + of_h) * own, name


def test_refusals(aa):
    Q, K, V, dH = make(1, 2, 4, 2, 8, 9, 64, "f32")
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    for bad in ((Q.double(), K, V), (Q, K.bfloat16(), V), (Q, K[:1], V), (Q, K, V[:, :, :5]), (Q[..., :32], K, V), (Q.cpu(), K, V),
                (Q, K.transpose(-1, -2).contiguous().transpose(-1, -2), V), (Q[0], K, V)):
        with pytest.raises((TypeError, ValueError)):
            aa.cross_forward(*bad)
    with pytest.raises(aa.AnchorAttnError):  # heads not a multiple of kv_heads
        aa.cross_forward(Q[:, :3], K, V)
    with pytest.raises(aa.AnchorAttnError):  # d
        aa.cross_forward(Q[..., :48].contiguous(), K[..., :48].contiguous(), V[..., :48].contiguous())
    with pytest.raises(aa.AnchorAttnError):
        aa.cross_forward(Q, K, V, scale=math.nan)
    with pytest.raises(aa.AnchorAttnError):  # H is Q
        aa.cross_forward(Q, K, V, H=Q)
    for bad in (torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError)):
            aa.cross_forward(Q, K, V, bad)
    with pytest.raises(ValueError):
        aa.cross_forward(Q, K, V, torch.zeros(3, dtype=torch.int32, device="cuda"))
    for bad in ((H[:, :2], lse, dH), (H, lse.double(), dH), (H, lse[:, :, :4], dH), (H, lse, dH.bfloat16())):
        with pytest.raises((TypeError, ValueError)):
            aa.cross_backward(Q, K, V, *bad)
    odd = torch.zeros(2 * 4 * 8 * 64 + 1, device="cuda")[1:].view(2, 4, 8, 64)  # not on 16 bytes
    with pytest.raises(aa.AnchorAttnError):
        aa.cross_forward(odd, K, V)
