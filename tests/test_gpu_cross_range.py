"""GPU: cross attention with scales of 0 and close to it."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.ops_reference import assert_within, cross_reference

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
