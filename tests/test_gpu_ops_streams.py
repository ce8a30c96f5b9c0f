"""GPU: a caller's output together with a stream of its own, in cross attention, rotation and the norm with it."""
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


def calls(aa, dtype):
    """{name: (the call with an output of its own and a stream, the shape of that output)}"""
    g = torch.Generator(device="cuda").manual_seed(3)
    Q, K, V = (torch.randn(2, h, n, 64, generator=g, device="cuda").to(dtype) for h, n in ((4, 300), (2, 500), (2, 500)))
    table = aa.rope_table(64)
    return {"cross_forward": lambda out, s: aa.cross_forward(Q, K, V, H=out, stream=s), "rope": lambda out, s: aa.rope(Q, table, out=out, stream=s),
            "norm_rope": lambda out, s: aa.norm_rope(Q, K, table, out=(out, None), stream=s)[0]}, Q


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["cross_forward", "rope", "norm_rope"])
def test_output_on_a_side_stream(aa, name, dtype):
    """The eager bits; and a buffer that the caller lets go of while the side stream is still to write it is not handed out."""
    all_, Q = calls(aa, dtype)
    call = all_[name]
    want = call(None, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.full_like(Q, 7.0)
    side.wait_stream(torch.cuda.current_stream())
    assert call(out, side).data_ptr() == out.data_ptr()
    side.synchronize()
    assert torch.equal(out, want)
    buf = torch.empty_like(Q)
    at = buf.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second
    call(buf, side)
    del buf
    other = [torch.empty_like(Q) for _ in range(4)]
    busy = not side.query()
    assert busy and all(t.data_ptr() != at for t in other)
    torch.cuda.synchronize()
