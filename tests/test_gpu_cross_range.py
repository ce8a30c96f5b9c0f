"""GPU: cross attention where scores are far outside of what fp32 tells apart, and scales of 0 and close to it."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.ops_reference import assert_within, cross_reference, half_step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# B, heads, kv_heads, n, s, d: one tile of states; row tiles in turn; a cluster's parts; parts joined by a second launch;
# CTAs without parts; a backward in parts
SHAPES = [(3, 2, 2, 40, 100, 64), (2, 4, 2, 30, 128, 128), (1, 2, 2, 150, 300, 64), (2, 4, 2, 300, 260, 128), (2, 8, 1, 1, 700, 128),
          (1, 1, 1, 1, 9000, 128), (40, 8, 4, 1, 900, 128), (1, 2, 1, 1500, 200, 64)]


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def make(seed, B, heads, kv, n, s, d, dtype, gain):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(by * torch.randn((B, h, rows, d), generator=g, device="cuda")).to(DT[dtype])
            for h, rows, by in ((heads, n, 1.5 * gain), (kv, s, gain), (kv, s, 1.0), (heads, n, 1.0))]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gain", [1e3, 1e4, 3e5])
@pytest.mark.parametrize("shape", SHAPES)
def test_far_scores(aa, dtype, gain, shape):
    """Scores of 10^6 to 10^11: a row's best state has the whole weight, and the gradients are within what P <= 1 allows."""
    B, heads, kv, n, s, d = shape
    Q, K, V, dH = make(31, *shape, dtype, gain)
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    assert bool(H.isfinite().all()) and bool(lse.isfinite().all())
    k, v, g = K.double().repeat_interleave(heads // kv, 1), V.double().repeat_interleave(heads // kv, 1), dH.double()
    x = (Q.double() @ k.mT) * d ** -0.5
    # scores are off by d roundings of fp32 of their products at the most: rows whose best state is ahead by more than that
    two = x.topk(2, -1)
    off = (d + 20) * 2.0 ** -23 * (Q.double().abs() @ k.abs().mT).amax(-1) * d ** -0.5
    sure = two.values[..., 0] - two.values[..., 1] > 40 + 2 * off
    assert float(sure.double().mean()) > 0.5
    best = v.gather(2, two.indices[..., :1].expand(*H.shape))
    # H = p v / p for one weight p, rounded once (bf16: half a step) before it meets v; the product, the quotient and H
    # are rounded once each
    assert bool(((H.double() - best).abs()[sure] <= (2 + 2.0 ** -6) * half_step(DT[dtype]) * best.abs()[sure] * (1 if dtype == "bf16" else 2)).all())
    assert bool(((lse.double() - two.values[..., 0]).abs()[sure] <= off[sure] + 2.0 ** -20 * two.values[..., 0].abs()[sure]).all())
    dQ, dK, dV = aa.cross_backward(Q, K, V, H, lse, dH)
    # P <= 1 and |dS| <= |dH . v| + |dH . H|, whatever lse's rounding makes of P; a hundredth for the roundings
    back = lambda t: t.unflatten(1, (kv, heads // kv)).sum(2)  # noqa: E731
    dS = (g @ v.mT).abs() + (g * H.double()).sum(-1, keepdim=True).abs()
    for got, most in ((dQ, d ** -0.5 * dS @ k.abs()), (dK, d ** -0.5 * back(dS.mT @ Q.double().abs())),
                      (dV, back(g.abs().sum(2, keepdim=True)).expand(V.shape))):
        assert bool((got.double().abs() <= 1.01 * most).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale,gain", [(0.0, 1e15), (2e-33, 1e16), (-1e-31, 1e15)])
@pytest.mark.parametrize("shape", SHAPES)
def test_small_scales(aa, dtype, scale, gain, shape):
    """Products of 10^31 and more: with a scale of 0 all states weigh alike, with a small one the scores count."""
    Q, K, V, dH = make(5, *shape, dtype, gain)
    L = torch.tensor([max(1, shape[4] - 37 * i) for i in range(shape[0])], dtype=torch.int32, device="cuda")
    H, lse = aa.cross_forward(Q, K, V, L, scale=scale, return_lse=True)
    ref = cross_reference(Q, K, V, L, scale, dH)
    assert_within(H, ref["H"], "H")
    assert_within(lse, ref["lse"], "lse")
    for name, got in zip(("dQ", "dK", "dV"), aa.cross_backward(Q, K, V, H, lse, dH, L, scale=scale)):
        assert_within(got, ref[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_no_scale_keeps_nan(aa, dtype, shape):
    """0 times a product that is no number is none; in its own row alone."""
    Q, K, V, _ = make(6, *shape, dtype, 1.0)
    H = aa.cross_forward(Q, K, V, scale=0.0)
    Q[0, 0, 0, 3] = math.nan
    H2 = aa.cross_forward(Q, K, V, scale=0.0)
    assert bool(H2[0, 0, 0].isnan().all())
    H2[0, 0, 0] = H[0, 0, 0]
    assert torch.equal(H, H2)
