"""GPU: which roundings the gradients of cross attention in bf16 carry where states are many."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("B,heads,kv,n,s", [(2, 4, 4, 300, 700), (1, 4, 2, 200, 1500), (1, 2, 2, 40, 3000), (1, 1, 1, 100, 4500)])
def test_dq_above_384_states(aa, d, B, heads, kv, n, s):
    """dS meets K as one bf16 number, in every fourth tile of 64 states (d = 16: every second) as two, counted from the first
    state, in a backward in parts too (the last two shapes).  Against dQ from a dS so rounded, in 64 bits with D from the H
    that the call is given, dQ is off by its own rounding.  Of the rest, fp32's, 2^-19 and less of dS, flips one rounding of
    dS in 2^10 by a whole step 2^-8: sqrt(2^-10 * 12) = 0.11 of a rounding, and sqrt(1 + 0.11^2) = 1.006.  Without the
    second number it would be off by sqrt(1 + 1 / 4) = 1.12 roundings; the bound lies between, with room for chance (4000
    elements and more)."""
    g = torch.Generator(device="cuda").manual_seed(s + d)
    Q, K, V, dH = ((torch.randn((B, h, rows, d), generator=g, device="cuda")).to(torch.bfloat16) for h, rows in ((heads, n), (kv, s), (kv, s), (heads, n)))
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    dQ = aa.cross_backward(Q, K, V, H, lse, dH)[0].double()
    q, k, v, h, up = (t.double() for t in (Q, K.repeat_interleave(heads // kv, 1), V.repeat_interleave(heads // kv, 1), H, dH))
    P = torch.softmax(q @ k.mT * d ** -0.5, -1)
    dS = P * (up @ v.mT - (up * h).sum(-1, keepdim=True))
    rounded = dS.to(torch.bfloat16).double()
    two = torch.arange(s, device="cuda") // 64 % (4 if d > 16 else 2) == 0
    want = d ** -0.5 * torch.where(two, dS, rounded) @ k
    own = float((want.to(torch.bfloat16).double() - want).norm())
    assert float((dQ - want).norm()) <= 1.04 * own
