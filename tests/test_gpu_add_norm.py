"""GPU: the norm of a residual sum, in 16, 32 and 8 bits, and its backward, against their definitions in 64 bits with bounds
that count the kernels' roundings (tests/decay_reference.py)."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.decay_reference import add_norm_backward_reference, add_norm_reference
from tests.ops_reference import F, assert_within, half_step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTHS = (16, 48, 64, 80, 256, 272, 512, 640, 768, 1008, 1024, 1040, 2048, 2064, 4096, 5008, 8192, 8208, 16384)


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def make(seed, shape, dtype, weight="same"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = lambda gain: (torch.randn(shape, generator=g, device="cuda") * gain).to(DT[dtype])  # noqa: E731
    w = None
    if weight != "none":
        w = (1 + 0.3 * torch.randn(shape[-1], generator=g, device="cuda")).to(torch.float32 if weight == "f32" else DT[dtype])
    return rows(1.0), rows(3.0), w, rows(1.0), rows(0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward(aa, dtype, D):
    for i, (rows, weight) in enumerate(((1, "same"), (5, "none"), (33, "f32"), (130, "same"))):
        X, R, w, *_ = make(i, (rows, D), dtype, weight)
        R = None if i == 1 else R
        S, (y, off) = add_norm_reference(X, R, w, 1e-5)
        Y, got = aa.add_norm(X, R, w, eps=1e-5)
        assert torch.equal(got, S) and (R is not None or got is X)
        assert_within(Y, (y, off + half_step(X.dtype) * y.abs()), f"{dtype} {rows} x {D}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("D", WIDTHS)
def test_8bit(aa, dtype, group, D):
    for i, rows in enumerate((1, 3, 70)):
        X, R, w, *_ = make(10 + i, (rows, D), dtype)
        if i == 2:
            X[5], R[5] = 0, 0
            X[6, : D // 2], R[6, : D // 2] = 0, 0
        S, (y, off) = add_norm_reference(X, R, w, 1e-6)
        Y, scales, got = aa.add_norm_8bit(X, R, w, group=group)
        size = group or D
        assert torch.equal(got, S) and Y.dtype == torch.float8_e4m3fn and scales.shape == (rows, -(-D // size))
        parts = y.abs().split(size, -1)
        top = torch.stack([p.amax(-1) for p in parts], -1)
        slack = torch.stack([p.amax(-1) for p in off.split(size, -1)], -1)
        assert_within(scales, (top / 448, slack / 448 + 2 * F * top / 448), "scales")
        over = scales.double().repeat_interleave(size, -1)[:, :D]
        # half a step of 2^-3 of the value, of 2^-9 (in scales) where it is subnormal; and fp32's
        assert_within(Y.double() * over, (y, 2.0 ** -4 * y.abs() + 2.0 ** -10 * over + 4 * (off + F * y.abs())), f"{dtype} {rows} x {D} group {group}")
        if i == 2:
            assert not scales[5].any() and not Y[5].float().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_backward(aa, dtype, D):
    for i, (rows, weight) in enumerate(((1, "same"), (37, "f32"), (130, "none"), (3000 if D < 2100 else 700, "same"))):
        X, R, w, dY, dS = make(20 + i, (rows, D), dtype, weight)
        dS = None if i == 1 else dS
        ref = add_norm_backward_reference(X, dY, w, dS, 1e-6)
        dX, dw = aa.add_norm_backward(X, dY, w, dS=dS)
        assert_within(dX, ref["dX"], f"{dtype} {rows} x {D}: dX")
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == w.dtype
            assert_within(dw, ref["dweight"], f"{dtype} {rows} x {D}: dweight")


def test_gradient_by_differences(aa):
    X, R, w, dY, dS = make(2, (6, 64), "f32")
    loss = lambda x, v: sum(float((a.double() * b.double()).sum()) for a, b in zip(aa.add_norm(x, R, v), (dY, dS)))  # noqa: E731
    Y, S = aa.add_norm(X, R, w)
    dX, dw = aa.add_norm_backward(S, dY, w, dS=dS)
    g = torch.Generator(device="cuda").manual_seed(5)
    h = 2.0 ** -6
    for name, grad, moved in (("X", dX, lambda t: loss(X + t, w)), ("weight", dw, lambda t: loss(X, w + t))):
        step = torch.randn(grad.shape, generator=g, device="cuda")
        want = (moved(h * step) - moved(-h * step)) / (2 * h)
        got = float((grad.double() * step.double()).sum())
        # the loss is rounded (about 2e-6 of its terms over 2 h), the difference is off by h^2 / 6 of a third derivative
        assert abs(got - want) <= 2e-3 * (1 + float(grad.norm() * step.norm())), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts(aa, dtype):
    """Views of wider buffers, batches, the sum over X or R, gradients over what they come from, no rows."""
    wide = [torch.randn(3, 40, 272, device="cuda").to(DT[dtype]) for _ in range(4)]
    X, R, dY, dS = (t[:, 2:39, 16:256] for t in wide)
    w = torch.rand(240, device="cuda").to(DT[dtype])
    dense = [t.contiguous() for t in (X, R, dY, dS)]
    Y, S = aa.add_norm(*dense[:2], w)
    assert Y.shape == (3, 37, 240)
    for a, b in zip(aa.add_norm(X, R, w), (Y, S)):
        assert torch.equal(a, b)
    flat = aa.add_norm(dense[0].reshape(-1, 240), dense[1].reshape(-1, 240), w)[0]
    assert torch.equal(flat.reshape(Y.shape), Y)
    Y8, scales, _ = aa.add_norm_8bit(*dense[:2], w, group=64)
    got = aa.add_norm_8bit(X, R, w, group=64)
    assert scales.shape == (3, 37, 4) and torch.equal(got[1], scales) and torch.equal(got[0].view(torch.uint8), Y8.view(torch.uint8))
    grads = aa.add_norm_backward(S, *dense[2:3], w, dS=dense[3])
    for a, b in zip(aa.add_norm_backward(S, dY, w, dS=dS), grads):
        assert torch.equal(a, b)
    for over in (0, 1):
        x = [t.clone() for t in dense[:2]]
        y, s = aa.add_norm(*x, w, S=x[over])
        assert s is x[over] and torch.equal(s, S) and torch.equal(y, Y) and torch.equal(x[1 - over], dense[1 - over])
    before = wide[1].clone()
    aa.add_norm(X, R, w, S=R)
    assert torch.equal(R, S)
    R.copy_(dense[1])
    assert torch.equal(wide[1], before)
    shared = dense[0][:1].expand(3, -1, -1)
    assert torch.equal(aa.add_norm(shared, R, w)[0], aa.add_norm(shared.contiguous(), R, w)[0])
    none = torch.empty(0, 64, device="cuda", dtype=DT[dtype])
    assert aa.add_norm(none, none)[0].shape == (0, 64) and aa.add_norm_8bit(none)[1].shape == (0, 1)
    w0 = torch.ones(64, device="cuda")
    assert not aa.add_norm_backward(none, none, w0)[1].any()


def test_extremes(aa):
    """Rows of tiny, huge and no numbers; an infinity or a NaN shows in its own row alone."""
    X = torch.randn(8, 256, device="cuda")
    X[0] *= 1e-30
    X[1] *= 1e18
    X[2], X[3, 7], X[4, 9] = 0, math.nan, math.inf
    w = torch.ones(256, device="cuda")
    Y, scales, _ = aa.add_norm_8bit(X, None, w, eps=0.0)
    y = X.double() / X.double().square().mean(-1, keepdim=True).sqrt()
    for r in (1, 5, 6, 7):
        assert_within(Y[r].double() * scales[r].double(), (y[r], 2.0 ** -4 * y[r].abs() + 2.0 ** -10 * scales[r].double() + 1e-6 * y[r].abs()), r)
    assert bool(Y[3].float().isnan().all()) and bool(scales[3].isnan().all()) and not bool(Y[5:].float().isnan().any())
    tiny = torch.full((1, 256), 1e-3, device="cuda")
    Y, scales, _ = aa.add_norm_8bit(tiny, None, torch.full((256,), 1e-38, device="cuda"), eps=1e-6)
    got = Y.double() * scales.double()
    # (scales below 2^-126 lose bits)
    want = 1e-38 * 1e-3 / math.sqrt(2e-6)
    assert float((got - want).abs().max()) <= 0.08 * want + 448 * 2.0 ** -149


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_on_a_stream_and_in_a_graph(aa, dtype):
    X, R, w, dY, dS = make(1, (700, 768), dtype)

    def run():
        return (*aa.add_norm(X, R, w), *aa.add_norm_backward(X, dY, w, dS=dS), *aa.add_norm_8bit(X, R, w, group=128))

    want = [t.clone() for t in run()]
    same = lambda a, b: torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a, b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [t.clone() for t in run()]
    side.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for t in out:
            t.zero_() if t.dtype == torch.float8_e4m3fn else t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(out, want))
