"""GPU: rotary positions and normalised rotary rows, forward and backward, against their definitions in 64 bits, with
bounds that count the kernels' roundings (tests/ops_reference.py)."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.ops_reference import assert_within, norm_rope_reference, rope_angles, rope_reference

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    return pkg


def rows(seed, B, heads, n, d, dtype, tokens=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (B, n, heads, d) if tokens else (B, heads, n, d)
    x = torch.randn(shape, generator=g, device="cuda").to(DT[dtype])
    return x.transpose(1, 2) if tokens else x


def positions_of(kind, B, n, axes=1):
    g = torch.Generator(device="cuda").manual_seed(n)
    if kind == "none":
        return None, torch.arange(n, device="cuda")[None, :, None].expand(1, n, axes)
    shape = (B, n, axes) if kind == "entry" else (n, axes)
    p = torch.randint(-1000, 10 ** 6, shape, generator=g, device="cuda", dtype=torch.int32 if n % 2 else torch.int64)
    full = p if kind == "entry" else p[None]
    return (p if axes > 1 else p[..., 0]).contiguous(), full


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (16, 2), (16, 6), (32, 32), (32, 12), (64, 64), (64, 32), (64, 26), (128, 128), (128, 64),
                                   (128, 48), (128, 126)])
def test_rope(aa, dtype, interleaved, d, rot):
    for i, (B, heads, n, kind) in enumerate(((1, 1, 1, "none"), (2, 3, 5, "shared"), (3, 5, 70, "entry"))):
        theta, magnitude = aa.rope_frequencies(rot)
        table = aa.rope_table(rot)
        X = rows(i, B, heads, n, d, dtype, tokens=i == 1)
        pos, full = positions_of(kind, B, n)
        angle = rope_angles(theta, full)
        assert_within(aa.rope(X, table, pos, interleaved=interleaved), rope_reference(X, angle, magnitude, interleaved), "Y")
        assert_within(aa.rope_backward(X, table, pos, interleaved=interleaved), rope_reference(X, angle, magnitude, interleaved, -1), "dX")


@pytest.mark.parametrize("how", [dict(scaling="linear", factor=8.0), dict(scaling="base", factor=4.0),
                                 dict(scaling="bands", factor=8.0, original=4096), dict(sections=(8, 8)), dict(sections=(4, 6, 6))])
def test_scaled_and_several_axes(aa, how):
    B, heads, n, d, rot = 2, 3, 41, 64, 32
    theta, magnitude = aa.rope_frequencies(rot, **how)
    table = aa.rope_table(rot, **how)
    X = rows(5, B, heads, n, d, "f32")
    for kind in ("none", "shared", "entry"):
        pos, full = positions_of(kind, B, n, len(theta))
        assert_within(aa.rope(X, table, pos), rope_reference(X, rope_angles(theta, full), magnitude, False), f"{how} {kind}")


def test_far_positions(aa):
    """At position 2^40 a double's angle is good to 1e-4 for the fastest pair; whole numbers give the exact one."""
    table = aa.rope_table(32)
    X = rows(6, 1, 2, 8, 32, "f32")
    start = 2 ** 40 + 12345
    got = aa.rope(X, table, start=start)
    turns = [[((start + i) * (int(p) % 2 ** 64) % 2 ** 64) / 2 ** 64 for p in table.phases[0].tolist()] for i in range(8)]
    angle = 2 * math.pi * torch.tensor(turns, dtype=torch.float64, device="cuda")[None]
    assert_within(got, rope_reference(X, angle, 1.0, False), "far")
    pos = torch.arange(start, start + 8, device="cuda")
    assert torch.equal(got, aa.rope(X, table, pos))
    # the same rows turned on by whole distances: positions p and p + 5 differ by a turn of 5 (relative positions)
    assert torch.equal(aa.rope(X, table, start=-3), aa.rope(X, table, torch.arange(-3, 5, device="cuda", dtype=torch.int32)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (32, 20), (64, 64), (64, 32), (128, 128), (128, 10), (128, 0)])
@pytest.mark.parametrize("weights", ["rows", "f32", "none"])
def test_norm_rope(aa, dtype, interleaved, d, rot, weights):
    eps = 1e-5
    for i, (B, heads, kv, n, s) in enumerate(((1, 1, 1, 1, 1), (2, 6, 2, 33, 70), (3, 2, 4, 300, 7))):
        theta, magnitude = aa.rope_frequencies(rot) if rot else ([[]], 1.0)
        table = aa.rope_table(rot) if rot else None
        Q, K = rows(i, B, heads, n, d, dtype, tokens=i == 1), rows(i + 9, B, kv, s, d, dtype, tokens=i == 2)
        dQ, dK = rows(i + 20, B, heads, n, d, dtype), rows(i + 21, B, kv, s, d, dtype, tokens=i == 1)
        wq, wk = (None if weights == "none" else (1 + 0.3 * torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(j), device="cuda"))
                  .to(DT[dtype] if weights == "rows" else torch.float32) for j in (1, 2))
        qp, qf = positions_of("entry", B, n)
        kp, kf = positions_of("shared", B, s)
        kp = kp.to(qp.dtype)
        how = dict(q_weight=wq, k_weight=wk, q_positions=qp, k_positions=kp, eps=eps, interleaved=interleaved)
        Y = aa.norm_rope(Q, K, table, **how)
        grads = aa.norm_rope_backward(Q, K, dQ, dK, table, **how)
        for j, (x, w, f, g) in enumerate(((Q, wq, qf, dQ), (K, wk, kf, dK))):
            angle = rope_angles(theta, f) if rot else torch.zeros(1, x.shape[2], 0, dtype=torch.float64, device="cuda")
            ref = norm_rope_reference(x, w, angle, magnitude, eps, interleaved, g)
            assert_within(Y[j], ref["Y"], f"Y{j}")
            assert_within(grads[j], ref["dX"], f"dX{j}")
            if w is None:
                assert grads[2 + j] is None
            else:
                assert grads[2 + j].dtype == w.dtype
                assert_within(grads[2 + j], ref["dw"], f"dw{j}")
        alone = aa.norm_rope(Q, None, table, q_weight=wq, q_positions=qp, eps=eps, interleaved=interleaved)
        assert alone[1] is None and torch.equal(alone[0], Y[0])
        back = aa.norm_rope_backward(Q, None, dQ, None, table, q_weight=wq, q_positions=qp, eps=eps, interleaved=interleaved)
        assert back[1] is None and back[3] is None and torch.equal(back[0], grads[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows_of_gradients(aa, dtype):
    """More rows than one wave of blocks: the weights' gradients are sums over all of them, the same bits each time."""
    B, heads, n, d = 2, 4, 9000, 64
    Q, dQ = rows(1, B, heads, n, d, dtype), rows(2, B, heads, n, d, dtype)
    w = torch.ones(d, device="cuda", dtype=torch.float32)
    table = aa.rope_table(d)
    theta, _ = aa.rope_frequencies(d)
    got = aa.norm_rope_backward(Q, None, dQ, None, table, q_weight=w)
    ref = norm_rope_reference(Q, w, rope_angles(theta, torch.arange(n, device="cuda")[None, :, None]), 1.0, 1e-6, False, dQ)
    assert_within(got[0], ref["dX"], "dX")
    assert_within(got[2], ref["dw"], "dw")
    again = aa.norm_rope_backward(Q, None, dQ, None, table, q_weight=w)
    assert torch.equal(got[0], again[0]) and torch.equal(got[2], again[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_parts_of_one_buffer(aa, dtype):
    """Queries and keys as parts of one token-major projection, turned where they lie; the values beside them stay."""
    B, n, heads, kv, d = 2, 50, 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    buf = torch.randn((B, n, heads + 2 * kv, d), generator=g, device="cuda").to(DT[dtype])
    q, k, v = (t.transpose(1, 2) for t in buf.split((heads, kv, kv), 2))
    table = aa.rope_table(d)
    want = aa.norm_rope(q, k, table)
    keep = v.clone()
    got = aa.norm_rope(q, k, table, out=(q, k))
    assert got[0].data_ptr() == buf.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)
    want = aa.rope(k, table, interleaved=True)
    aa.rope(k, table, interleaved=True, out=k)
    assert torch.equal(k, want) and torch.equal(v, keep)
    buf = torch.randn((B, n, kv, 3, d), generator=g, device="cuda").to(DT[dtype])  # the parts of a head next to one another
    q2, k2, v2 = (buf[:, :, :, i].transpose(1, 2) for i in range(3))
    want, keep = aa.norm_rope(q2, k2, table), v2.clone()
    aa.norm_rope(q2, k2, table, out=(q2, k2))
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1]) and torch.equal(v2, keep)
    with pytest.raises(aa.AnchorAttnError):  # an output over the other tensor
        aa.norm_rope(q, k, table, out=(q, q[:, :kv]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_pass_through(aa, dtype):
    """Columns behind rot and rows beside a bad one are not touched by infinities or NaN."""
    X = rows(3, 1, 2, 20, 64, dtype)
    table = aa.rope_table(20)
    want = aa.rope(X, table)
    assert torch.equal(want[..., 20:], X[..., 20:])
    X2 = X.clone()
    X2[0, 0, 3, 25], X2[0, 1, 4, 0] = math.inf, math.nan
    got = aa.rope(X2, table)
    assert float(got[0, 0, 3, 25]) == math.inf and torch.equal(got[0, 0, 3, :20], want[0, 0, 3, :20])
    assert int(got.isnan().sum()) == 2
    w = torch.ones(64, device="cuda", dtype=DT[dtype])
    zero = torch.zeros_like(X)
    for t in aa.norm_rope_backward(zero, None, X, None, table, q_weight=w)[::2]:
        assert bool(t.isfinite().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_streams_and_graphs(aa, dtype):
    table = aa.rope_table(32)
    w = torch.ones(64, device="cuda", dtype=DT[dtype])
    for B, heads, n in ((0, 2, 3), (2, 0, 3), (2, 2, 0)):
        X = rows(1, B, heads, n, 64, dtype)
        assert aa.rope(X, table).shape == X.shape
        got = aa.norm_rope_backward(X, None, X, None, table, q_weight=w)
        assert bool((got[2] == 0).all())
    X, G = rows(2, 2, 4, 700, 64, dtype), rows(3, 2, 4, 700, 64, dtype)
    step = lambda stream=None: [t for t in (*aa.norm_rope(X, G, table, q_weight=w, stream=stream), *aa.norm_rope_backward(  # noqa: E731
        X, G, G, X, table, q_weight=w, k_weight=w, stream=stream))]
    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = step(st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_gradient_against_differences(aa):
    X, G = rows(1, 1, 2, 7, 32, "f32"), rows(2, 1, 2, 7, 32, "f32")
    table = aa.rope_table(32)
    w = 1 + 0.1 * torch.randn(32, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    dX, _, dw, _ = aa.norm_rope_backward(X, None, G, None, table, q_weight=w)
    for i, grad in enumerate((dX, dw)):
        step = torch.randn(grad.shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
        loss = []
        for e in (-1, 1):
            x, y = (X + e * 2.0 ** -7 * step, w) if i == 0 else (X, w + e * 2.0 ** -7 * step)
            loss.append(float((aa.norm_rope(x, None, table, q_weight=y)[0].double() * G.double()).sum()))
        want = float((grad.double() * step.double()).sum())
        # 448 values off by 1e-7 each, times 2^6, and the third derivative times h^2
        assert abs((loss[1] - loss[0]) * 2.0 ** 6 - want) <= 5e-3 * (1 + abs(want))


def test_refusals(aa):
    X = rows(1, 2, 3, 5, 64, "f32")
    table = aa.rope_table(32)
    p = torch.arange(5, device="cuda")
    for call in (lambda: aa.rope(X.double(), table), lambda: aa.rope(X, None), lambda: aa.rope(X, (table.phases.int(), 1.0)),
                 lambda: aa.rope(X, table, p[:4]), lambda: aa.rope(X, table, p.float()), lambda: aa.rope(X, table, p.cpu()),
                 lambda: aa.rope(X, table, p[None].expand(2, 5)), lambda: aa.rope(X.transpose(2, 3), table),
                 lambda: aa.rope(X, table, out=X.bfloat16()), lambda: aa.rope(X, aa.RopeTable(table.phases.cpu())),
                 lambda: aa.norm_rope(X, X.bfloat16(), table), lambda: aa.norm_rope(X, X[..., :32], table),
                 lambda: aa.norm_rope(X, None, table, q_weight=torch.ones(32, device="cuda")),
                 lambda: aa.norm_rope(X, None, table, q_weight=torch.ones(64, device="cuda", dtype=torch.bfloat16)),
                 lambda: aa.norm_rope_backward(X, None, X[:1], None, table)):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: aa.rope(X[..., :48].contiguous(), table), lambda: aa.norm_rope(X, None, table, eps=-1.0),
                 lambda: aa.rope(X, (table.phases, math.inf)), lambda: aa.rope(X[..., :16], table),
                 lambda: aa.rope(X, table, out=X.as_strided(X.shape, (0, 0, 64, 1))), lambda: aa.rope(X[:, 1:], table, out=X[:, :2])):
        with pytest.raises(aa.AnchorAttnError):
            call()
