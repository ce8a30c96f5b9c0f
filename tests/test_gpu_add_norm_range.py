"""GPU: the norm of a residual sum for rows whose squares leave fp32's range, from its smallest numbers to its largest, with eps = 0 too."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.decay_reference import add_norm_backward_reference, add_norm_reference
from tests.ops_reference import F, assert_within, half_step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# rows of numbers between half and one and a half of a power of two; None: zeros
POWERS = (0, -126, -148, 126, None, -100, 64, 3, -75, 63, -62, 100, 62, -40, None, 40, -50, -51, 110, -132, 1)
WIDTHS = (16, 48, 256, 768, 1024, 1040, 2048, 4096, 8208, 16384)
LEAST = 2.0 ** -149  # a step of the smallest numbers


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def make(seed, D, dtype, powers=POWERS):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = len(powers)
    size = torch.tensor([0.0 if p is None else 2.0 ** p for p in powers], dtype=torch.float64, device="cuda")[:, None]
    sign = torch.randint(0, 2, (n, D), generator=g, device="cuda") * 2 - 1
    X = ((torch.rand(n, D, generator=g, device="cuda").double() + 0.5) * sign * size).to(DT[dtype])
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(DT[dtype])
    dY, dS = (torch.randn(n, D, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    return X, w, dY, dS


def definition(S, w, eps):
    """The norm in 64 bits (zeros of a row of zeros) and what fp32 may be off by."""
    _, (y, off) = add_norm_reference(S, None, w, eps)
    zero = (S == 0).all(-1, keepdim=True)
    return y.masked_fill(zero, 0), off.masked_fill(zero, 0) + 4 * LEAST


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -101, 2.0 ** -20, 2.0 ** 100])
def test_forward(aa, dtype, eps):
    for i, D in enumerate(WIDTHS):
        X, w, *_ = make(i, D, dtype)
        y, off = definition(X, w, eps)
        Y, S = aa.add_norm(X, None, w, eps=eps)
        assert S is X
        assert_within(Y, (y, off + half_step(X.dtype) * y.abs()), f"{D}")
        # half of X twice is X (but where a half is rounded: the smallest numbers)
        half = (X.float() / 2).to(X.dtype)
        Y, S = aa.add_norm(half, half, w, eps=eps)
        assert torch.equal(S, (half.float() * 2).to(X.dtype))
        y, off = definition(S, w, eps)
        assert_within(Y, (y, off + half_step(X.dtype) * y.abs()), f"{D}, a sum")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_8bit(aa, dtype, group):
    for i, D in enumerate(WIDTHS):
        X, w, *_ = make(20 + i, D, dtype)
        y, off = definition(X, w, 0.0)
        Y, scales, _ = aa.add_norm_8bit(X, None, w, eps=0.0, group=group)
        size = group or D
        over = scales.double().repeat_interleave(size, -1)[:, :D]
        assert_within(Y.double() * over, (y, 2.0 ** -4 * y.abs() + 2.0 ** -10 * over + 4 * (off + F * y.abs())), f"{D}")
        zero = (X == 0).all(-1)
        assert not scales[zero].any() and not Y[zero].float().any() and bool((scales[~zero] > 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -20])
def test_backward(aa, dtype, eps):
    for i, D in enumerate(WIDTHS):
        # (gradients of rows below 2^-120 pass the type's largest number)
        powers = [p for p in POWERS if p is None or p > -120 or eps > 1e-9]
        X, w, dY, dS = make(40 + i, D, dtype, powers)
        some = (X != 0).any(-1)
        for more in (None, dS):
            dX, dw = aa.add_norm_backward(X, dY, w, dS=more, eps=eps)
            ref = add_norm_backward_reference(X[some], dY[some], w, None if more is None else more[some], eps)
            if eps > 0:
                dw_ref = add_norm_backward_reference(X, dY, w, more, eps)["dweight"]
            else:
                dw_ref = ref["dweight"]
            assert_within(dX[some], (ref["dX"][0], ref["dX"][1] + 4 * LEAST), f"{D}: dX")
            assert_within(dw, dw_ref, f"{D}: dweight")
            if eps == 0:
                assert torch.equal(dX[~some], torch.zeros_like(dX[~some]) if more is None else more[~some])


def test_gradients_that_pass_the_largest_number(aa):
    # rows of the smallest numbers: 1 / sqrt(mean) counts as the largest fp32 number where it passes it, so that the row's part of dweight is
    # smaller than it were, and dX infinite at most; other rows do not suffer
    X, w, dY, _ = make(3, 256, "f32", (-148, 0, -140))
    dX, dw = aa.add_norm_backward(X, dY, w, eps=0.0)
    ref = add_norm_backward_reference(X[1:2], dY[1:2], w, None, 0.0)
    assert not bool(dX.isnan().any())
    assert_within(dX[1:2], ref["dX"], "dX")
    # hat is at most 2^128 times the numbers, 1.5 x 2^-140 and 2^-147.4
    assert_within(dw, (ref["dweight"][0], ref["dweight"][1] + 1.5 * 2.0 ** -12 * dY.abs().amax(0).double() + 2.0 ** -19 * dY.abs().amax(0).double()), "dweight")
    true = add_norm_backward_reference(X, dY, w, None, 0.0)["dX"][0]
    big = dX.abs() > 1e38
    assert bool(big[[0, 2]].any()) and torch.equal(dX.sign()[big], true.float().sign()[big])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 768, 4096])
def test_infinities_stay_in_their_rows(aa, dtype, D):
    X, w, dY, _ = make(6, D, dtype, (0, 0, 64, 0, -70, 0, 0, 0))
    bad = X.clone()
    bad[1, 5], bad[3, 7], bad[6] = math.inf, math.nan, -math.inf
    good = [0, 2, 4, 5, 7]
    for eps in (0.0, 1e-6):
        want, got = aa.add_norm(X, None, w, eps=eps)[0], aa.add_norm(bad, None, w, eps=eps)[0]
        assert torch.equal(got[good], want[good])
        assert bool(got[1, 5].isnan()) and bool(got[3].isnan().all()) and bool(got[6].isnan().all())
        Y, scales, _ = aa.add_norm_8bit(bad, None, w, eps=eps)
        assert bool(scales[[1, 3, 6]].isnan().all()) and bool(scales[good].isfinite().all())
        want, got = aa.add_norm_backward(X, dY, w, eps=eps)[0], aa.add_norm_backward(bad, dY, w, eps=eps)[0]
        assert torch.equal(got[good], want[good]) and bool(got[[3, 6]].isnan().all())


def test_a_number_far_above_the_others(aa):
    # one column carries the row's size; the others are what is left of them
    X, w, dY, _ = make(8, 768, "f32", (0, -60, -140, 30))
    X[:, 100] = torch.tensor([2.0 ** 100, 2.0 ** 64, 2.0 ** -60, 2.0 ** 127], device="cuda")
    y, off = definition(X, w, 0.0)
    assert_within(aa.add_norm(X, None, w, eps=0.0)[0], (y, off + F * y.abs()), "Y")
    ref = add_norm_backward_reference(X, dY, w, None, 0.0)
    dX, dw = aa.add_norm_backward(X, dY, w, eps=0.0)
    assert_within(dX, (ref["dX"][0], ref["dX"][1] + 8 * LEAST), "dX")
    assert_within(dw, (ref["dweight"][0], ref["dweight"][1] + 8 * LEAST), "dweight")
