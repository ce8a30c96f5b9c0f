"""GPU: the operators together, as a layer uses them: queries and an encoder's keys out of token-major projections,
normalised and turned where they lie, cross attention and its gradients, and the anchor attention on the same turned
queries; a training step against the formulas in 64 bits, and a token of a decoder against the whole sequence."""
import math

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


def definition(Q, K, V, wq, wk, theta, L, start):
    """H in 64 bits, differentiable."""
    def turned(x, w, at):
        z = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a = torch.arange(at, at + x.shape[2], device=x.device, dtype=torch.float64)[:, None] * theta
        p, q = z.chunk(2, -1)
        return torch.cat([p * a.cos() - q * a.sin(), p * a.sin() + q * a.cos()], -1)

    group = Q.shape[1] // K.shape[1]
    q, k, v = turned(Q, wq, start), turned(K, wk, 0).repeat_interleave(group, 1), V.repeat_interleave(group, 1)
    off = torch.arange(K.shape[2], device=Q.device)[None, :] >= L[:, None]
    return torch.softmax((q @ k.mT * Q.shape[3] ** -0.5).masked_fill(off[:, None, None], -math.inf), -1) @ v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_training_step(aa, dtype, d):
    B, heads, kv, n, s = 2, 6, 2, 210, 333
    g = torch.Generator(device="cuda").manual_seed(d)
    make = lambda rows, h: torch.randn(B, rows, h, d, generator=g, device="cuda").to(dtype)  # noqa: E731
    q_proj, kv_proj, up = make(n, heads), make(s, 2 * kv), make(n, heads)
    Q, dH = q_proj.transpose(1, 2), up.transpose(1, 2)
    K, V = (t.transpose(1, 2) for t in kv_proj.split(kv, 2))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    L = torch.tensor([s, 100], dtype=torch.int32, device="cuda")
    table = aa.rope_table(d)
    how = dict(q_weight=wq, k_weight=wk, q_start=5)
    Qr, Kr = aa.norm_rope(Q, K, table, **how)
    H, lse = aa.cross_forward(Qr, Kr, V, L, return_lse=True)
    dQr, dKr, dV = aa.cross_backward(Qr, Kr, V, H, lse, dH, L)
    dQ, dK, dwq, dwk = aa.norm_rope_backward(Q, K, dQr, dKr, table, **how)
    theta = torch.tensor(aa.rope_frequencies(d)[0][0], dtype=torch.float64, device="cuda")
    x = [t.double().requires_grad_(True) for t in (Q, K, V, wq, wk)]
    ref = definition(*x, theta, L, 5)
    ref.backward(dH.double())
    # bf16: the chain rounds Q', K', P, H, dS, dQ' and dQ, half a step of 2^-8 at the most each, and a 2-norm adds at the
    # most eight of them; fp32: sums of some hundred products
    tol = 8 * 2.0 ** -8 if dtype == torch.bfloat16 else 400 * 2.0 ** -24
    for name, got, want in (("H", H, ref), ("dQ", dQ, x[0].grad), ("dK", dK, x[1].grad), ("dV", dV, x[2].grad), ("dwq", dwq, x[3].grad),
                            ("dwk", dwk, x[4].grad)):
        assert got.shape == want.shape
        rel = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert rel <= tol, (name, rel, tol)


@pytest.mark.parametrize("d", [64, 128])
def test_a_token_at_a_time(aa, d):
    """A decoder's tokens one by one, each turned to its place, give the rows of the whole sequence."""
    B, heads, kv, n, s = 3, 8, 2, 20, 700
    g = torch.Generator(device="cuda").manual_seed(d)
    Q = torch.randn(B, heads, n, d, generator=g, device="cuda").to(torch.bfloat16)
    K, V = (torch.randn(B, kv, s, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    L = torch.tensor([700, 0, 300], dtype=torch.int32, device="cuda")
    table = aa.rope_table(d, scaling="bands", factor=4.0, original=4096)
    Qr, Kr = aa.norm_rope(Q, K, table, q_start=100)
    whole = aa.cross_forward(Qr, Kr, V, L)
    for i in range(n):
        row, _ = aa.norm_rope(Q[:, :, i:i + 1], None, table, q_start=100 + i)
        assert torch.equal(row, Qr[:, :, i:i + 1])
        one = aa.cross_forward(row, Kr, V, L)
        # the same weights and states, summed in other parts: two roundings of P and one of H on either side
        off = (one.double() - whole[:, :, i:i + 1].double()).norm() / whole[:, :, i:i + 1].double().norm()
        assert float(off) <= 6 * 2.0 ** -8
    assert bool((whole[1] == 0).all())


def test_turned_queries_into_the_anchor_attention(aa):
    """The rows that norm_rope leaves are what forward and causal_forward take: image positions on two axes, anchors normed."""
    B, heads, n, m, d = 2, 3, 196, 40, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    Q, V = (torch.randn(B, heads, n, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    U = torch.randn(heads, m, d, generator=g, device="cuda").to(torch.bfloat16)
    at = torch.stack([torch.arange(n, device="cuda") // 14, torch.arange(n, device="cuda") % 14], -1)
    Qr, _ = aa.norm_rope(Q, None, aa.rope_table(d, sections=(16, 16)), q_positions=at)
    Ur = aa.norm_rope(U[None], None, None)[0][0]
    q, u, v = Qr.double(), Ur.double(), V.double()
    A = torch.softmax(q @ u.mT * d ** -0.5, -1)
    want = A @ ((A.mT @ v) / A.sum(-2)[..., None])
    assert bool(((aa.forward(Qr, Ur, V).double() - want).abs() <= 1e-2 + 2e-2 * want.abs()).all())
    assert bool((aa.causal_forward(Qr, Ur, V)[:, :, -1].double() - want[:, :, -1]).abs().max() <= 3e-2)
