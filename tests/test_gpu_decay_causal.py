"""GPU: attention with decaying states: which rows a NaN or an infinity at one token reaches, and what a call that gives the states out changes."""
import math

import pytest
import torch

from tests.conftest import gpu_available
from tests.ops_reference import half_step

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = {"bf16": 128, "f32": 64}


@pytest.fixture(scope="module")
def aa():
    import linear_complexity_anchor_gb300 as pkg
    pkg.load()
    yield pkg
    assert pkg.device_error() == 0


def make(seed, B, heads, n, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = {name: torch.randn(B, heads, n, d, generator=g, device="cuda").to(DT[dtype]) for name in ("Q", "K", "V", "dH")}
    x["rate"] = -1.0 / torch.linspace(20, 900, heads, device="cuda")
    x["state"], x["dstate"] = (torch.randn(B, heads, d, d, generator=g, device="cuda") for _ in range(2))
    return x


def run(aa, x):
    H, last = aa.decay_forward(x["Q"], x["K"], x["V"], x["rate"], state=x["state"], return_state=True)
    dQ, dK, dV, first = aa.decay_backward(x["Q"], x["K"], x["V"], x["dH"], x["rate"], state=x["state"], dstate=x["dstate"])
    return {"H": H, "last": last, "dQ": dQ, "dK": dK, "dV": dV, "first": first}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,heads,n,d", [(2, 2, 450, 64), (1, 2, 1500, 32), (160, 1, 300, 64), (2, 2, 450, 128), (1, 1, 1500, 128)])
def test_a_bad_token(aa, dtype, B, heads, n, d):
    # H and dQ of the tokens before it stay as they are, but for those of its chunk; so do dK and dV of the tokens behind it; own rows alone where
    # the token is a row of the result; other heads and entries altogether.
    size = CHUNK[dtype]
    x = make(d, B, heads, n, d, dtype)
    want = run(aa, x)
    forward = {"Q": ("own", None, "back", "back"), "K": ("ahead", "ahead", None, "own"), "V": ("ahead", "ahead", "own", None), "dH": (None, "own", "back", "back")}
    for j in (0, size + 3, n - 1):
        for name, reach in forward.items():
            for bad in (math.nan, -math.inf):
                y = {**x, name: x[name].clone()}
                y[name][B - 1, heads - 1, j, d // 2] = bad
                got = run(aa, y)
                for out, how in zip(("H", "dQ", "dK", "dV"), reach):
                    ok = torch.zeros(n, dtype=torch.bool, device="cuda")  # rows that may differ
                    if how == "own":
                        ok[j] = True
                    elif how == "ahead":
                        ok[j // size * size:] = True
                    elif how == "back":
                        ok[:(j // size + 1) * size] = True
                    same = (got[out] == want[out]).all(-1)
                    same[B - 1, heads - 1, ok] = True
                    assert bool(same.all()), (name, j, bad, out)
                    if how:  # it shows where it counts
                        assert not bool(got[out][B - 1, heads - 1, j].isfinite().all()), (name, j, bad, out)
                for out, touched in (("last", name in "KV"), ("first", name in ("Q", "dH"))):
                    same = (got[out] == want[out]).all(-1).all(-1)
                    assert bool(same.flatten()[:-1].all()) and bool(same.flatten()[-1]) != touched, (name, j, bad, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,heads,n,d", [(2, 3, 700, 64), (1, 2, 3000, 128), (160, 1, 300, 64)])
def test_giving_the_states_out(aa, dtype, B, heads, n, d):
    # In bf16 the states that go into H have one rounding fewer where they are given out, so that single bits of H may differ: by a rounding of the result,
    # and by what half a step of X~ is of it.  In fp32 they are the same bits.
    x = make(5, B, heads, n, d, dtype)
    a = aa.decay_forward(x["Q"], x["K"], x["V"], x["rate"], state=x["state"])
    b, _ = aa.decay_forward(x["Q"], x["K"], x["V"], x["rate"], state=x["state"], return_state=True)
    if dtype == "f32":
        assert torch.equal(a, b)
    else:
        u = half_step(a.dtype)
        assert float((a.double() - b.double()).norm() / b.double().norm()) < u
        assert torch.equal(b, aa.decay_forward(x["Q"], x["K"], x["V"], x["rate"], state=x["state"], return_state=True)[0])
