"""CPU: what the entries of attention with decaying states and of the norm of a residual sum refuse before they touch a
device, which streams their tensors are recorded on, and what the binding checks.  Addresses are made up and never read."""
import contextlib
import ctypes
import math
import struct

import pytest
import torch

import linear_complexity_anchor_gb300 as aa
from linear_complexity_anchor_gb300 import _decay, _norm, _views
from tests.test_ops_abi import A, ALIAS, INVALID, UNSUPPORTED, F, I, P, View, dense
from tests.test_ops_streams import Library, Stream, expect

ALLOC = 4
N = 4000  # tokens, in segments


class Decay(ctypes.Structure):
    _fields_ = [(n, I) for n in ("dtype", "B", "heads", "n", "d")] + [("scale", F)] + [
        (n, View) for n in ("Q", "K", "V", "H", "dH", "dQ", "dK", "dV")] + [
        (n, P) for n in ("log_decay", "lengths", "state", "last", "dlast", "dstate")]


class Step(ctypes.Structure):
    _fields_ = [(n, I) for n in ("dtype", "B", "heads", "n", "d", "slot_count")] + [("scale", F)] + [
        (n, View) for n in ("Q", "K", "V", "H")] + [(n, P) for n in ("log_decay", "states", "slots")]


class AddNorm(ctypes.Structure):
    _fields_ = [(n, I) for n in ("dtype", "B", "n", "D", "weight_f32", "bits8", "group")] + [("eps", F)] + [
        (n, View) for n in ("X", "R", "S", "Y", "dY", "dS", "dX")] + [("weight", P), ("dweight", P), ("scales", P)]


@pytest.fixture(scope="module")
def lib():
    from linear_complexity_anchor_gb300 import _build
    _build.build()
    return aa.load()


def test_packed_sizes(lib):
    v = _views.VIEW
    assert struct.calcsize("=5if" + 8 * v + "6Q") == ctypes.sizeof(Decay)
    assert struct.calcsize("=6if4x" + 4 * v + "3Q") == ctypes.sizeof(Step)
    assert struct.calcsize("=7if" + 7 * v + "QQQ") == ctypes.sizeof(AddNorm)
    assert len(_decay._pack(*[0] * 5, 0.0, *[0] * 38)) == ctypes.sizeof(Decay)
    assert len(_decay._pack_step(*[0] * 6, 0.0, *[0] * 19)) == ctypes.sizeof(Step)
    assert len(_norm._pack(*[0] * 7, 0.0, *[0] * 31)) == ctypes.sizeof(AddNorm)


def decay(lib, backward=False, **change):
    z = dict(dtype=0, B=2, heads=4, n=N, d=64, scale=0.125)
    z.update({k: v for k, v in change.items() if k in z})
    p = Decay(**z)
    for i, name in enumerate(("Q", "K", "V", "H", "dH", "dQ", "dK", "dV")):
        setattr(p, name, dense(A * (i + 1), z["heads"], z["n"], z["d"]))
    for i, name in enumerate(("log_decay", "lengths", "state", "last", "dlast", "dstate")):
        setattr(p, name, A * (20 + i))
    for k, v in change.items():
        if k not in z:
            setattr(p, k, v)
    return (lib.anchor_attn_decay_backward if backward else lib.anchor_attn_decay_forward)(ctypes.byref(p), None)


@pytest.mark.parametrize("backward", [False, True])
def test_decay_refusals(lib, backward, monkeypatch):
    monkeypatch.setenv("ANCHOR_ATTN_TEST_FAIL_ALLOC", "1")  # what gets past the checks ends at the workspace
    c = lambda **kw: decay(lib, backward, **kw)  # noqa: E731
    assert c() == ALLOC and c(state=0, lengths=0, last=0, dlast=0, dstate=0) == ALLOC
    for name in ("dtype", "B", "heads", "n"):
        assert c(**{name: -1}) == INVALID
    assert c(dtype=2) == INVALID and c(d=48) == UNSUPPORTED and c(d=0) == UNSUPPORTED and c(d=256) == UNSUPPORTED
    assert c(scale=math.inf) == INVALID and c(scale=math.nan) == INVALID
    assert c(n=1 << 29) == UNSUPPORTED and c(B=1 << 23, n=1) == UNSUPPORTED and c(B=1 << 14, heads=1 << 10, n=200) == UNSUPPORTED
    assert c(log_decay=0) == INVALID and c(log_decay=A * 20 + 2) == INVALID and c(lengths=A * 21 + 1) == INVALID
    for name in ("state", "last", "dlast", "dstate"):
        assert c(**{name: A * 40 + 4}) == INVALID
    for name in ("Q", "K", "V") + (("dH", "dQ", "dK", "dV") if backward else ("H",)):
        at = A * 50
        assert c(**{name: View(0, 1, 1, 1)}) == INVALID
        assert c(**{name: View(at + 8, 4 * N * 64, N * 64, 64)}) == INVALID
        assert c(**{name: View(at, 4 * N * 64, N * 64, 68)}) == INVALID
        assert c(**{name: View(at, 4 * N * 64, N * 64, 32)}) == INVALID
        assert c(**{name: View(at, -4 * N * 64, N * 64, 64)}) == INVALID
        assert c(**{name: View(at, 1 << 45, N * 64, 64)}) == INVALID
        assert c(**{name: View(at, 4 * N * 64, 0, 64)}) == (ALLOC if name in ("Q", "K", "V", "dH") else INVALID)
    size = 2 * 4 * N * 64 * 2
    for out, at in (("dQ", 6), ("dK", 7), ("dV", 8)) if backward else (("H", 4),):
        for other in (1, 2, 3) + ((5,) if backward else ()):
            assert c(**{out: dense(A * other, 4, N, 64)}) == ALIAS and c(**{out: dense(A * other + size - 128, 4, N, 64)}) == ALIAS
        for name in ("log_decay", "lengths", "state", "dlast" if backward else "last"):
            assert c(**{name: A * at + 64}) == ALIAS
    if backward:
        assert c(dQ=dense(7 * A, 4, N, 64)) == ALIAS and c(dV=dense(6 * A + 128, 4, N, 64)) == ALIAS
        assert c(dstate=A * 24) == ALIAS and c(dstate=A * 22) == ALIAS and c(dstate=A * 5) == ALIAS and c(dstate=A * 8) == ALIAS
    else:
        assert c(last=A * 22) == ALIAS and c(last=A * 20) == ALIAS and c(last=A) == ALIAS
    assert c(B=0) == 0 and c(heads=0) == 0 and c(n=0, last=0, dstate=0) == 0
    assert lib.anchor_attn_decay_forward(None, None) == INVALID and lib.anchor_attn_decay_backward(None, None) == INVALID


def step(lib, **change):
    z = dict(dtype=0, B=2, heads=4, n=1, d=64, slot_count=5, scale=0.125)
    z.update({k: v for k, v in change.items() if k in z})
    p = Step(**z)
    for i, name in enumerate(("Q", "K", "V", "H")):
        setattr(p, name, dense(A * (i + 1), z["heads"], z["n"], z["d"]))
    p.log_decay, p.states, p.slots = A * 20, A * 21, A * 22
    for k, v in change.items():
        if k not in z:
            setattr(p, k, v)
    return lib.anchor_attn_decay_step(ctypes.byref(p), None)


def test_step_refusals(lib):
    c = lambda **kw: step(lib, **kw)  # noqa: E731
    for name in ("dtype", "B", "heads", "n", "slot_count"):
        assert c(**{name: -1}) == INVALID
    assert c(dtype=2) == INVALID and c(d=24) == UNSUPPORTED and c(scale=math.nan) == INVALID
    assert c(slots=0, slot_count=1) == INVALID and c(states=0) == INVALID and c(states=A * 21 + 8) == INVALID
    assert c(log_decay=0) == INVALID and c(slots=A * 22 + 2) == INVALID and c(B=1 << 24) == UNSUPPORTED
    assert c(Q=View(0, 1, 1, 1)) == INVALID and c(H=View(A * 4 + 4, 256, 64, 64)) == INVALID and c(H=View(A * 4, 256, 0, 64)) == INVALID
    assert c(H=dense(A, 4, 1, 64)) == ALIAS and c(H=dense(21 * A + 4096, 4, 1, 64)) == ALIAS and c(H=dense(22 * A, 4, 1, 64)) == ALIAS
    assert c(K=dense(21 * A, 4, 1, 64)) == ALIAS and c(states=A * 20) == ALIAS and c(states=A * 22) == ALIAS
    assert c(B=0) == 0 and c(heads=0) == 0 and c(n=0) == 0
    assert lib.anchor_attn_decay_step(None, None) == INVALID


def add_norm(lib, backward=False, **change):
    z = dict(dtype=0, B=2, n=8, D=64, weight_f32=0, bits8=0, group=0, eps=1e-6)
    z.update({k: v for k, v in change.items() if k in z})
    p = AddNorm(**z)
    for i, name in enumerate(("X", "R", "S", "Y", "dY", "dS", "dX")):
        setattr(p, name, View(A * (i + 1), z["n"] * z["D"], 0, z["D"]))
    p.weight, p.dweight, p.scales = A * 20, A * 21 if backward else 0, A * 22
    for k, v in change.items():
        if k not in z:
            setattr(p, k, v)
    return (lib.anchor_attn_add_norm_backward if backward else lib.anchor_attn_add_norm)(ctypes.byref(p), None)


@pytest.mark.parametrize("backward", [False, True])
def test_add_norm_refusals(lib, backward, monkeypatch):
    monkeypatch.setenv("ANCHOR_ATTN_TEST_FAIL_ALLOC", "1")
    c = lambda **kw: add_norm(lib, backward, **kw)  # noqa: E731
    for bad in (dict(dtype=2), dict(B=-1), dict(n=-1), dict(weight_f32=2), dict(bits8=-1), dict(group=16), dict(group=-32), dict(eps=-1.0),
                dict(eps=math.nan), dict(eps=math.inf), dict(weight=A * 20 + 4), dict(scales=A * 22 + 2), dict(dweight=A * 21 + 2)):
        assert c(**bad) == INVALID, bad
    for D in (0, 8, 20, 16400, -16):
        assert c(D=D) == UNSUPPORTED
    assert c(B=1 << 15, n=1 << 16) == UNSUPPORTED
    for name in ("S", "dY", "dX") if backward else ("X", "Y", "S"):
        assert c(**{name: View(0, 512, 0, 64)}) == INVALID
        assert c(**{name: View(A * 30 + 8, 512, 0, 64)}) == INVALID and c(**{name: View(A * 30, 512, 0, 68)}) == INVALID
        assert c(**{name: View(A * 30, 512, 0, 48)}) == INVALID and c(**{name: View(A * 30, -512, 0, 64)}) == INVALID
    at = lambda k, more=0: View(A * k + more, 512, 0, 64)  # noqa: E731
    if backward:
        assert c(bits8=1) == INVALID
        assert c() == ALLOC and c(dS=View(0, 0, 0, 0)) == ALLOC
        assert c(dX=at(5)) == ALLOC and c(dX=at(6)) == ALLOC and c(dX=at(3)) == ALIAS and c(dX=at(5, 128)) == ALIAS
        assert c(dX=at(20)) == ALIAS and c(dX=at(21)) == ALIAS and c(dweight=A * 3) == ALIAS and c(dweight=A * 20) == ALIAS and c(dweight=A * 6) == ALIAS
    else:
        assert c(dweight=A * 21) == INVALID and c(bits8=1, scales=0) == INVALID
        assert c(Y=at(1)) == ALIAS and c(Y=at(2)) == ALIAS and c(Y=at(3)) == ALIAS and c(S=at(1, 128)) == ALIAS and c(S=at(4)) == ALIAS
        assert c(Y=at(20)) == ALIAS and c(bits8=1, scales=A) == ALIAS and c(bits8=1, scales=A * 4) == ALIAS and c(bits8=1, scales=A * 20) == ALIAS
        assert c(bits8=1, Y=View(A * 4, 520, 0, 64)) == INVALID
        assert c(B=0) == 0 and c(n=0) == 0
    assert lib.anchor_attn_add_norm(None, None) == INVALID and lib.anchor_attn_add_norm_backward(None, None) == INVALID


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
    for module in (_decay, _norm):
        monkeypatch.setattr(module, "library", Library)
    return now, side, found


@pytest.mark.parametrize("given", [False, True])
def test_streams(seen, given):
    now, side, found = seen
    Q, K, V, dH, out = (torch.zeros(2, 4, 5, 16) for _ in range(5))
    g, L = torch.zeros(4), torch.ones(2, dtype=torch.int32)
    state, dstate, pool = torch.zeros(2, 4, 16, 16), torch.zeros(2, 4, 16, 16), torch.zeros(3, 4, 16, 16)
    H, last = aa.decay_forward(Q, K, V, g, L, state=state, H=out if given else None, return_state=True, stream=side)
    expect(found, [(t, side) for t in (Q, K, V, g, L, state)] + ([(H, side)] if given else []), [(last, now)] + ([] if given else [(H, now)]))
    found.clear()
    grads = aa.decay_backward(Q, K, V, dH, g, L, state=state, dstate=dstate, stream=side)
    expect(found, [(t, side) for t in (Q, K, V, dH, g, L, state, dstate)], [(t, now) for t in grads])
    found.clear()
    H = aa.decay_step(Q, K, V, g, pool, L, H=out if given else None, stream=side)
    expect(found, [(t, side) for t in (Q, K, V, g, pool, L)] + ([(H, side)] if given else []), [] if given else [(H, now)])
    found.clear()
    X, R, S0, dY, dS = (torch.zeros(3, 16) for _ in range(5))
    w = torch.ones(16)
    Y, S = aa.add_norm(X, R, w, S=S0 if given else None, stream=side)
    assert (S is S0) == given
    expect(found, [(t, side) for t in (X, R, w)] + ([(S, side)] if given else []), [(Y, now)] + ([] if given else [(S, now)]))
    found.clear()
    Y, scales, _ = aa.add_norm_8bit(X, None, w, stream=side)
    expect(found, [(X, side), (w, side)], [(Y, now), (scales, now)])
    found.clear()
    dX, dw = aa.add_norm_backward(S, dY, w, dS=dS, stream=side)
    expect(found, [(t, side) for t in (S, dY, w, dS)], [(dX, now), (dw, now)])


def test_binding_refusals(seen):
    side = seen[1]
    Q = torch.zeros(2, 4, 5, 16)
    g, state = torch.zeros(4), torch.zeros(2, 4, 16, 16)
    for bad, kind in ((dict(log_decay=None), TypeError), (dict(log_decay=g.double()), TypeError), (dict(log_decay=torch.zeros(3)), ValueError),
                      (dict(lengths=torch.ones(2)), TypeError), (dict(lengths=torch.ones(3, dtype=torch.int32)), ValueError),
                      (dict(state=state.half()), TypeError), (dict(state=state.mT), ValueError), (dict(state=state[:1]), ValueError),
                      (dict(K=Q[:, :2]), ValueError), (dict(V=Q.bfloat16()), TypeError), (dict(Q=Q.half()), TypeError),
                      (dict(Q=Q[0]), ValueError), (dict(H=Q[:1]), ValueError), (dict(K=[1]), TypeError)):
        how = {**dict(Q=Q, K=Q, V=Q, log_decay=g), **bad}
        with pytest.raises(kind):
            aa.decay_forward(**how, stream=side)
    with pytest.raises(ValueError):
        aa.decay_backward(Q, Q, Q, Q[:, :, :4], g, stream=side)
    with pytest.raises(TypeError):
        aa.decay_backward(Q, Q, Q, Q, g, dstate=state.double(), stream=side)
    for bad, kind in ((dict(states=state[0]), TypeError), (dict(states=state[:, :3]), ValueError), (dict(slots=torch.zeros(2)), TypeError),
                      (dict(slots=torch.zeros(3, dtype=torch.int32)), ValueError), (dict(states=None), TypeError)):
        with pytest.raises(kind):
            aa.decay_step(**{**dict(Q=Q, K=Q, V=Q, log_decay=g, states=state), **bad}, stream=side)
    X = torch.zeros(3, 16)
    for bad, kind in ((dict(X=X.half()), TypeError), (dict(R=X.bfloat16()), TypeError), (dict(R=X[:2]), ValueError), (dict(X=X[0]), ValueError),
                      (dict(X=X.T), ValueError), (dict(weight=torch.ones(8)), ValueError), (dict(weight=torch.ones(16).double()), TypeError),
                      (dict(weight=1.0), TypeError), (dict(S=X), ValueError), (dict(X=None), TypeError)):
        with pytest.raises(kind):
            aa.add_norm(**{**dict(X=X), **bad}, stream=side)
    with pytest.raises(ValueError):
        aa.add_norm_8bit(X, group=16, stream=side)
    with pytest.raises(ValueError):
        aa.add_norm_backward(X, X[:2], stream=side)
