"""GPU: attention with decaying states over rows that lie more than 2^31 elements apart within one head."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,step", [(3, 3 << 29), (20, 1 << 27), (150, 1 << 24)])
def test_far_rows(aa, dtype, n, step):
    # token by token, in one chunk, in two: heads beside one another, tokens far apart
    heads, d = 2, 64
    assert (n - 1) * step > 1 << 31
    buf = torch.empty((n - 1) * step + heads * d, dtype=DT[dtype], device="cuda")
    far = buf.as_strided((1, heads, n, d), (0, d, step, 1))
    g = torch.Generator(device="cuda").manual_seed(n)
    near = [torch.randn(1, heads, n, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(4)]
    rate = torch.tensor([-0.01, -0.2], device="cuda")
    want, grads = aa.decay_forward(*near[:3], rate), aa.decay_backward(*near, rate)[:3]
    for i in range(4):  # each of Q, K, V, dH in its turn
        far.copy_(near[i])
        x = [far if j == i else t for j, t in enumerate(near)]
        if i < 3:
            assert torch.equal(aa.decay_forward(*x[:3], rate), want)
        for a, b in zip(aa.decay_backward(*x, rate)[:3], grads):
            assert torch.equal(a, b)
    far.zero_()
    aa.decay_forward(*near[:3], rate, H=far)
    assert torch.equal(far, want)
    states = torch.zeros(1, heads, d, d, device="cuda")
    steps = aa.decay_step(*near[:3], rate, states.clone())
    far.copy_(near[1])
    assert torch.equal(aa.decay_step(near[0], far, near[2], rate, states.clone()), steps)
    far.zero_()
    aa.decay_step(*near[:3], rate, states.clone(), H=far)
    assert torch.equal(far, steps)
