"""GPU: what is left of a state behind many tokens that add nothing, exp(length log_decay) of it: the factors of chunks and of segments
are rounded, and what a rounding leaves must not add up over them."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F = 2.0 ** -24


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def left(aa, dtype, B, heads, n, d, rate, lengths, X):
    """The last state of a forward, and the first state's gradient of a backward, of tokens of zeros."""
    zero = torch.zeros(1, 1, n, d, device="cuda", dtype=DT[dtype]).expand(B, heads, n, d)
    last = aa.decay_forward(zero, zero, zero, rate, lengths, state=X, return_state=True)[1]
    first = aa.decay_backward(zero, zero, zero, zero, rate, lengths, state=X, dstate=X)[3]
    return last, first


def off_by(got, X, rate, lengths):
    """The relative error of each entry's head: in the root of the mean square, and of the mean."""
    want = X.double() * torch.exp(lengths.double()[:, None] * rate.double()[None])[..., None, None]
    return ((got - want).square().sum((2, 3)) / want.square().sum((2, 3))).sqrt()


def rounded(chunks):
    """`chunks` roundings to nearest of numbers that do not go together: f / sqrt(12) to f / sqrt(3) each (by where the number lies between powers of
    two), in the root of the mean square; four times that for the spread, and two roundings that all numbers of a head share."""
    return 4 * (chunks / 12) ** 0.5 * F + 2 * F


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_that_end_inside_a_chunk(aa, dtype):
    # Entries of one segment (as many heads as there are places), whose last chunk, of 128 rows or of 64, is the 31st, 32nd or 64th, whole and not.
    lengths = [31 * 128 + 1, 31 * 128 + 42, 32 * 128, 31 * 128, 30 * 128 + 7, 32 * 128 + 1, 63 * 128 + 100, 64 * 128 - 1, 64 * 128, 33 * 128 + 5,
               31 * 64 + 1, 31 * 64 + 21, 32 * 64, 31 * 64, 63 * 64 + 5, 63 * 64 + 63, 64 * 64 + 1, 95 * 64 + 30, 127 * 64 + 33]
    B, heads, n, d = len(lengths), 32, 64 * 128, 64
    assert B * heads >= 4 * 152
    L = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    rate = -1.0 / torch.logspace(2.8, 5, heads, device="cuda")
    X = torch.randn(B, heads, d, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    chunks = torch.ceil(L / (128.0 if dtype == "bf16" else 64.0))
    bound = torch.tensor([rounded(c) for c in chunks.tolist()], device="cuda")[:, None]
    for got in left(aa, dtype, B, heads, n, d, rate, L, X):
        off = off_by(got, X, rate, L)
        assert bool((off < bound).all()), (off / bound).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens(aa, dtype):
    # token by token: one rounding a token, whether a token takes much or little
    heads, n, d = 16, 512, 32
    X = torch.randn(1, heads, d, d, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    rate = -torch.logspace(-4.5, -1.6, heads, device="cuda")
    zero, states = torch.zeros(1, heads, n, d, device="cuda", dtype=DT[dtype]), X.clone()
    aa.decay_step(zero, zero, zero, rate, states)
    off = off_by(states, X, rate, torch.tensor([n], device="cuda"))
    assert off.max().item() < rounded(2 * n), (off / rounded(2 * n))
