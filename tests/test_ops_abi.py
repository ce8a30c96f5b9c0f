"""CPU: what the cross attention and rotary entries of the C ABI refuse before they touch a device, and the tables of
frequencies.  Addresses are made up and never read: every call here ends in a refusal or has nothing to do."""
import ctypes
import math

import pytest

INVALID, UNSUPPORTED, ALIAS = 1, 2, 3
A = 1 << 32


I, F, L, P = ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_void_p


class View(ctypes.Structure):
    _fields_ = [("ptr", P), ("batch", L), ("head", L), ("row", L)]


class Cross(ctypes.Structure):
    _fields_ = [(n, I) for n in ("dtype", "B", "heads", "kv_heads", "n", "s", "d")] + [("scale", F)] + [
        (n, View) for n in ("Q", "K", "V", "H", "dH", "dQ", "dK", "dV")] + [("lse", P), ("lengths", P)]


class Rope(ctypes.Structure):
    _fields_ = [(n, I) for n in ("dtype", "d", "rot", "axes", "interleaved", "norm", "weight_f32", "positions64")] + [
        ("eps", F), ("magnitude", F), ("phases", P)]


class Rows(ctypes.Structure):
    _fields_ = [(n, View) for n in ("X", "Y", "dY", "dX")] + [("weight", P), ("dweight", P), ("positions", P), ("positions_batch", L),
                                                              ("start", L), ("B", I), ("heads", I), ("n", I)]


def test_packed_sizes(pkg):
    """What the binding packs is as long as the structures."""
    import struct
    from linear_complexity_anchor_gb300._views import VIEW
    assert struct.calcsize("=" + VIEW) == ctypes.sizeof(View) == 32
    assert struct.calcsize("=7if" + 8 * VIEW + "QQ") == ctypes.sizeof(Cross)
    assert struct.calcsize("=8i2fQ") == ctypes.sizeof(Rope)
    assert struct.calcsize("=" + 4 * VIEW + "QQQqq3i4x") == ctypes.sizeof(Rows)


@pytest.fixture(scope="module")
def pkg():
    from linear_complexity_anchor_gb300 import _build
    _build.build()
    import linear_complexity_anchor_gb300 as p
    p.load()
    return p


def dense(at, heads, n, d):
    return View(at, heads * n * d, n * d, d)


def cross(pkg, backward=False, **change):
    z = dict(dtype=0, B=2, heads=4, kv_heads=2, n=8, s=16, d=64, scale=0.125)
    z.update({k: v for k, v in change.items() if k in z})
    p = Cross(**z)
    for i, name in enumerate(("Q", "K", "V", "H", "dH", "dQ", "dK", "dV")):
        q = name in ("Q", "H", "dH", "dQ")
        setattr(p, name, dense(A * (i + 1), z["heads"] if q else z["kv_heads"], z["n"] if q else z["s"], z["d"]))
    p.lse, p.lengths = A * 20, A * 21
    for k, v in change.items():
        if k not in z:
            setattr(p, k, v)
    fn = pkg.load().anchor_attn_cross_backward if backward else pkg.load().anchor_attn_cross_forward
    return fn(ctypes.byref(p), None)


@pytest.mark.parametrize("backward", [False, True])
def test_cross_refusals(pkg, backward):
    c = lambda **kw: cross(pkg, backward, **kw)  # noqa: E731
    for name in ("dtype", "B", "heads", "kv_heads", "n", "s"):
        assert c(**{name: -1}) == INVALID
    assert c(dtype=2) == INVALID and c(d=48) == UNSUPPORTED and c(d=0) == UNSUPPORTED
    assert c(heads=3) == INVALID and c(kv_heads=0) == INVALID and c(scale=math.inf) == INVALID
    assert c(n=1 << 30) == UNSUPPORTED and c(B=1 << 28, n=64) == UNSUPPORTED
    assert c(B=1 << 29, heads=2, kv_heads=2, n=1, s=0) == UNSUPPORTED
    assert c(Q=View(0, 1, 1, 1)) == INVALID
    assert c(Q=View(A + 8, 2048, 512, 64)) == INVALID          # base not on 16 bytes
    assert c(K=View(2 * A, 2048, 1024, 68)) == INVALID         # stride not of 16 bytes
    assert c(V=View(3 * A, -2048, 1024, 64)) == INVALID
    assert c(K=View(2 * A, 1 << 45, 1024, 64)) == INVALID      # beyond any memory
    assert c(lengths=A + 2) == INVALID and c(lse=A * 20 + 2) == INVALID
    if backward:
        assert c(lse=0) == INVALID
        assert c(dK=dense(A + 64, 2, 16, 64)) == ALIAS and c(dK=dense(8 * A, 2, 16, 64)) == ALIAS
        assert c(dQ=View(6 * A, 0, 512, 64)) == INVALID        # written rows on one another
        assert c(dV=View(8 * A, 2048, 1024, 32)) == INVALID
        assert c(dQ=dense(20 * A, 4, 8, 64)) == ALIAS
    else:
        assert c(H=dense(A, 4, 8, 64)) == ALIAS and c(H=dense(2 * A + 16, 4, 8, 64)) == ALIAS
        assert c(H=View(4 * A, 0, 512, 64)) == INVALID and c(lse=A + 16) == ALIAS and c(lse=21 * A) == ALIAS
    # nothing to do
    assert c(B=0) == 0 and c(heads=0, kv_heads=0) == 0
    assert c(n=0, s=0) == 0
    assert pkg.load().anchor_attn_cross_forward(None, None) == INVALID


def rope(pkg, backward=False, second=False, how={}, **change):
    h = Rope(dtype=0, d=64, rot=64, axes=1, interleaved=0, norm=1, weight_f32=0, positions64=0, eps=1e-6, magnitude=1.0, phases=A * 30)
    for k, v in how.items():
        setattr(h, k, v)
    z = dict(B=2, heads=4, n=8)
    z.update({k: v for k, v in change.items() if k in z})

    def rows(base):
        r = Rows(**z)
        for i, name in enumerate(("X", "Y", "dY", "dX")):
            setattr(r, name, dense(base + A * (i + 1), z["heads"], z["n"], 64))
        r.weight, r.positions, r.positions_batch = A * 31, A * 32, 8
        return r

    r, r2 = rows(0), rows(10 * A)
    for k, v in change.items():
        if k not in z:
            setattr(r2 if second else r, k, v)
    fn = pkg.load().anchor_attn_norm_rope_backward if backward else pkg.load().anchor_attn_norm_rope
    return fn(ctypes.byref(h), ctypes.byref(r), ctypes.byref(r2) if second else None, None)


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_refusals(pkg, backward, second):
    c = lambda how={}, **kw: rope(pkg, backward, second, how, **kw)  # noqa: E731
    for bad in (dict(dtype=2), dict(interleaved=2), dict(norm=-1), dict(weight_f32=3), dict(positions64=2), dict(rot=-2), dict(rot=3),
                dict(rot=66), dict(axes=0), dict(axes=4), dict(eps=-1.0), dict(eps=math.nan), dict(magnitude=math.inf), dict(phases=0),
                dict(phases=A + 4)):
        assert c(bad) == INVALID, bad
    assert c(dict(d=48)) == UNSUPPORTED
    assert c(B=-1) == INVALID and c(heads=-1) == INVALID and c(n=-1) == INVALID and c(positions_batch=-1) == INVALID
    assert c(B=1 << 15, n=1 << 16) == UNSUPPORTED
    assert c(positions=A + 2) == INVALID and c(dict(positions64=1), positions=A + 4) == INVALID and c(weight=A + 1) == INVALID
    out, read = ("dX", "dY") if backward else ("Y", "X")
    assert c(**{out: View(0, 1, 1, 1)}) == INVALID and c(**{read: View(0, 1, 1, 1)}) == INVALID
    assert c(**{out: View(A * 5 + 4, 2048, 512, 64)}) == INVALID and c(**{read: View(A * 5, 2048, 512, 60)}) == INVALID
    assert c(**{out: View(A * 5, 2048, 0, 64)}) == INVALID
    assert c(**{out: dense(A * 31 - 64, 4, 8, 64)}) == ALIAS and c(**{out: dense(A * 30, 4, 8, 64)}) == ALIAS
    assert c(**{out: dense(A * 32, 4, 8, 64)}) == ALIAS
    at = 11 * A if second else A
    assert c(**{out: dense(at + 1024, 4, 8, 64)}) == ALIAS             # partly over X
    if backward:
        assert c(dX=dense(at, 4, 8, 64)) == ALIAS
        assert c(dweight=A * 31) == ALIAS and c(dweight=at) == ALIAS
        assert c(dict(norm=0), dweight=A * 40) == INVALID
    else:
        assert c(dweight=A * 40) == INVALID
    if second:  # an output over the other tensor's
        assert c(**{out: dense((4 if backward else 2) * A, 4, 8, 64)}) == ALIAS
    elif not backward:
        assert c(B=0) == 0 and c(heads=0) == 0 and c(n=0) == 0
    # parts of one token-major buffer do not meet; parts that share a head do
    buf = lambda first: View(50 * A + first * 128, 8 * 8 * 64, 64, 8 * 64)  # noqa: E731
    assert c(dict(eps=-1.0), **{out: buf(0), read: buf(4)}) == INVALID
    assert c(**{out: buf(0), read: buf(3)}) == ALIAS


def test_parts_of_one_buffer(pkg, monkeypatch):
    """Which parts of one buffer count as overlapping, in every order of the axes that a projection's output has: what gets
    past the checks ends at the workspace, which the environment refuses."""
    ALLOC = 4
    monkeypatch.setenv("ANCHOR_ATTN_TEST_FAIL_ALLOC", "1")
    d, n, H = 64, 8, 4
    call = lambda dX, dY: rope(pkg, True, False, {}, dX=dX, dY=dY, dweight=A * 40)  # noqa: E731
    # [B, n, part, head, d], [B, n, head, part, d], [B, part, head, n, d], [part, B, head, n, d]: batch, head, row, part
    for sb, sh, sn, part in ((3 * H * n * d, d, 3 * H * d, H * d), (3 * H * n * d, 3 * d, 3 * H * d, d),
                             (3 * H * n * d, n * d, d, H * n * d), (H * n * d, n * d, d, 2 * H * n * d)):
        at = lambda k, more=0: View(50 * A + 2 * (part * k + more), sb, sh, sn)  # noqa: E731
        for i in range(3):
            for j in range(3):
                assert call(at(i), at(j)) == (ALIAS if i == j else ALLOC), (sb, sh, sn, part, i, j)
            assert call(at(i, 8), at(i)) == ALIAS
    # heads of one tensor over those of the next
    assert call(View(50 * A + 2 * 3 * d, 2 * H * n * d, d, 2 * H * d), View(50 * A, 2 * H * n * d, d, 2 * H * d)) == ALIAS


def test_rope_frequencies(pkg):
    theta, magnitude = pkg.rope_frequencies(8, 10000.0)
    assert magnitude == 1.0 and theta == [[1.0, pytest.approx(0.1), pytest.approx(0.01), pytest.approx(0.001)]]
    assert pkg.rope_frequencies(8, scaling="linear", factor=4.0)[0][0][1] == pytest.approx(0.025)
    base = pkg.rope_frequencies(8, scaling="base", factor=4.0)[0][0]
    assert base[0] == 1.0 and base[3] == pytest.approx(0.001 / 4)
    bands, magnitude = pkg.rope_frequencies(64, scaling="bands", factor=16.0, original=4096)
    plain = pkg.rope_frequencies(64)[0][0]
    for t, p in zip(bands[0], plain):
        turns = 4096 * p / (2 * math.pi)
        g = min(1.0, max(0.0, (turns - 1) / 31))
        assert t == pytest.approx(p * g + p / 16 * (1 - g), rel=1e-12)
    assert bands[0][0] == plain[0] and bands[0][-1] == pytest.approx(plain[-1] / 16) and magnitude == pytest.approx(0.1 * math.log(16) + 1)
    two, _ = pkg.rope_frequencies(16, sections=(4, 4))
    assert two[0] == [1.0, pytest.approx(0.1), pytest.approx(0.01), pytest.approx(0.001), 0, 0, 0, 0] and two[1][4:] == two[0][:4]
    table = pkg.rope_table(8, device="cpu")
    assert [int(p) for p in table.phases[0]] == [round(t / (2 * math.pi) * 2 ** 64) for t in theta[0]]
    assert table.phases.shape == (1, 4) and table.magnitude == 1.0
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=-1.0), dict(rot=8, factor=0.0), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="bands"), dict(rot=8, sections=(2, 1)), dict(rot=8, sections=(4, 0)), dict(rot=2, scaling="base"),
                dict(rot=8, sections=(1, 1, 1, 1))):
        with pytest.raises(ValueError):
            pkg.rope_frequencies(**bad)
