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
@pytest.mark.parametrize("heads,n", [(1, 32768), (1, 131072), (3, 50021), (1, 9999)])
def test_over_segments(aa, dtype, heads, n):
    # A few heads: up to 256 segments.  The walk along them is one rounding of its result; the last segment's chunks one each: at most 25 (of
    # 3200 rows: 3 heads of 50021 bf16 tokens, backward).
    d = 64
    X = torch.randn(1, heads, d, d, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
    L = torch.full((1,), n, dtype=torch.int32, device="cuda")
    worst = 0.0
    for part in (0.1, 0.35, 0.8, 1.7, 3.1, 6.0):
        rate = torch.full((heads,), -part / n, device="cuda") * torch.linspace(1, 1.1, heads, device="cuda")
        for got in left(aa, dtype, 1, heads, n, d, rate, L, X):
            worst = max(worst, off_by(got, X, rate, L).max().item())
    assert worst < rounded(25), (worst, rounded(25))


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
@pytest.mark.parametrize("d", [16, 128])
def test_other_widths(aa, dtype, d):
    # Segments of 896 rows at most: fourteen chunks of 64.  Four of these at 3 / 3977 are factors below e^-1/2, of which nothing is carried: each
    # is off by a step of its own (expf's error: one unit in the last place, 2 f of a number above 1/2) that all numbers share.
    for heads, n in ((1, 20000), (5, 31 * 128 + 9)):
        X = torch.randn(1, heads, d, d, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda")
        L = torch.full((1,), n, dtype=torch.int32, device="cuda")
        rate = -torch.linspace(0.3, 3.0, heads, device="cuda") / n
        for got in left(aa, dtype, 1, heads, n, d, rate, L, X):
            off = off_by(got, X, rate, L)
            assert off.max().item() < rounded(14) + 4 * 2 * F, (heads, off)


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
