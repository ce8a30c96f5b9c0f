"""GPU: the workspaces that are kept between calls, and how they are given back."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def test_release_workspaces():
    """A workspace of 256 MB stays after its call, goes back when asked for, and the next call takes it anew."""
    import linear_complexity_anchor_gb300 as aa
    g = torch.Generator(device="cuda").manual_seed(1)
    Q, dH = (torch.randn(64, 64, 16384, 16, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    K, V = (torch.randn(64, 64, 8, 16, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    H, lse = aa.cross_forward(Q, K, V, return_lse=True)
    aa.release_workspaces()

    def step():
        return aa.cross_backward(Q, K, V, H, lse, dH)

    def used():
        torch.cuda.synchronize()
        free, total = torch.cuda.mem_get_info()
        return total - free - torch.cuda.memory_reserved()

    want = step()
    got = step()  # (torch keeps the memory of the results of both)
    before = used()
    aa.release_workspaces()
    after = used()
    assert before - after >= 64 * 64 * 16384 * 4  # D alone, fp32, a row
    aa.release_workspaces()
    assert used() == after
    del got
    for a, b in zip(want, step()):
        assert torch.equal(a, b)
    assert used() >= after + 64 * 64 * 16384 * 4
    aa.release_workspaces()
    assert aa.device_error() == 0
