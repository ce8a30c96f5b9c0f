"""CPU: the largest sizes that cross attention takes.  Addresses are made up and never read: what gets past the checks ends
at the workspace, which the environment refuses."""
import pytest

from tests.test_ops_abi import UNSUPPORTED, View, cross, pkg  # noqa: F401

ALLOC = 4
MOST = 2 ** 31 - 1024  # of B * heads * (n + s)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,heads,kv", [(1, 1, 1), (1, 4, 2), (1, 8, 1)])
@pytest.mark.parametrize("many", ["n", "s"])
def test_largest_sizes(pkg, monkeypatch, dtype, B, heads, kv, many):  # noqa: F811
    """Tile counts and the walks over them add up to a few tiles to a size: 2^31 less 1024 is the most."""
    monkeypatch.setenv("ANCHOR_ATTN_TEST_FAIL_ALLOC", "1")

    def call(total, backward=True):
        few = 8
        size = {"n": few, "s": few, many: total // (B * heads) - few}
        views = {}
        for i, name in enumerate(("Q", "K", "V", "H", "dH", "dQ", "dK", "dV")):
            rows = size["n"] if name in ("Q", "H", "dH", "dQ") else size["s"]
            views[name] = View((i + 1) << 44, 0, rows * 16, 16)
        return cross(pkg, backward, dtype=dtype, B=B, heads=heads, kv_heads=kv, d=16, lse=20 << 44, lengths=21 << 44, **size, **views)

    assert call(MOST) == ALLOC
    for more in (1, 512, 1023):
        total = MOST + more * B * heads
        if total < 2 ** 31 + B * heads:
            assert call(total) == UNSUPPORTED
            assert call(total, backward=False) == UNSUPPORTED


def test_nothing_to_release(pkg):  # noqa: F811
    """Without a workspace there is no pool, and no device is touched."""
    assert pkg.load().anchor_attn_release_workspaces() == 0 and pkg.release_workspaces() is None
