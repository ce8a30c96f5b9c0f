"""CPU: which streams the calls that take views name to the allocator for each tensor, with a library, streams and CUDA
tensors that are stood in for: nothing here touches a device."""
import contextlib

import pytest
import torch

import linear_complexity_anchor_gb300 as aa
from linear_complexity_anchor_gb300 import _cross, _rope, _views


class Stream:
    def __init__(self, handle):
        self.device, self.cuda_stream = torch.device("cuda", 0), handle


class Library:
    """Every call succeeds and writes nothing."""
    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def seen(monkeypatch):
    """(the current stream, a side stream, what was recorded as {data_ptr: [streams]})"""
    now, side, found = Stream(1), Stream(2), {}
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: found.setdefault(t.data_ptr(), []).append(s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(_views, "_current_device", lambda: 0)
    for module in (_cross, _rope):
        monkeypatch.setattr(module, "library", Library)
    return now, side, found


def rows(heads, n):
    return torch.zeros(2, heads, n, 16)


def expect(found, on_side, on_now):
    assert {p: s for p, s in found.items()} == {**{t.data_ptr(): [s] for t, s in on_side}, **{t.data_ptr(): [s] for t, s in on_now}}


@pytest.mark.parametrize("given", [False, True])
def test_cross(seen, given):
    """A caller's H is written on the side stream, so that its memory may not be handed out before that is done; an H made
    by the call is the side stream's own, and the caller's to use on the current one."""
    now, side, found = seen
    Q, K, V, dH, out = rows(4, 5), rows(2, 7), rows(2, 7), rows(4, 5), rows(4, 5)
    L = torch.ones(2, dtype=torch.int32)
    H, lse = aa.cross_forward(Q, K, V, L, H=out if given else None, return_lse=True, stream=side)
    assert (H is out) == given
    expect(found, [(t, side) for t in (Q, K, V, L)] + ([(H, side)] if given else []), [(lse, now)] + ([] if given else [(H, now)]))
    found.clear()
    grads = aa.cross_backward(Q, K, V, H, lse, dH, L, stream=side)
    expect(found, [(t, side) for t in (Q, K, V, H, lse, dH, L)], [(t, now) for t in grads])
    found.clear()
    aa.cross_forward(Q, K, V, L, H=out, stream=now)
    assert not found


@pytest.mark.parametrize("given", [(), (0,), (1,), (0, 1)])
def test_norm_rope(seen, given):
    now, side, found = seen
    Q, K, dQ, dK, to = rows(4, 5), rows(2, 7), rows(4, 5), rows(2, 7), (rows(4, 5), rows(2, 7))
    w, p = torch.ones(16), torch.arange(5)
    table = aa.rope_table(16, device="cpu")
    out = tuple(to[i] if i in given else None for i in range(2))
    got = aa.norm_rope(Q, K, table, q_weight=w, q_positions=p, out=out, stream=side)
    expect(found, [(t, side) for t in (Q, K, w, p, table.phases)] + [(got[i], side) for i in given], [(got[i], now) for i in range(2) if i not in given])
    found.clear()
    made = [t for t in aa.norm_rope_backward(Q, K, dQ, dK, table, q_weight=w, q_positions=p, stream=side) if t is not None]
    expect(found, [(t, side) for t in (Q, K, dQ, dK, w, p, table.phases)], [(t, now) for t in made])


@pytest.mark.parametrize("given", [False, True])
def test_rope(seen, given):
    now, side, found = seen
    X, out, table = rows(4, 5), rows(4, 5), aa.rope_table(16, device="cpu")
    got = aa.rope(X, table, out=out if given else None, stream=side)
    expect(found, [(X, side), (table.phases, side)] + ([(got, side)] if given else []), [] if given else [(got, now)])
    found.clear()
    got = aa.rope_backward(X, table, stream=side)
    expect(found, [(X, side), (table.phases, side)], [(got, now)])
    found.clear()
    aa.rope(X, table, out=X, stream=side)  # in place
    assert set(found) == {X.data_ptr(), table.phases.data_ptr()} and all(s is side for t in found.values() for s in t)
