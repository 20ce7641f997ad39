"""CPU checks of the draft-verification entry points: refusals that need no device, and the host part of the
rotary plan against its formulas."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def osc():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_decode_gb300 as o
    return o


def test_null_cache_is_refused(osc):
    lib, bad = osc.lib(), osc.ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.oscar_build_tables(None, 1, None, None, None, 0, None, None, None, None, None, None, None, 0, None) == bad
    assert lib.oscar_tree_layout(None, 1, 4, None, None, None, None, None, None) == bad
    assert lib.oscar_tree_workspace_bytes(None, 1, 4, 0, ctypes.byref(n)) == bad
    assert lib.oscar_tree_attention(None, 0, 1, 4, None, None, None, None, None, None, None, 0, None, 0.1, None, 0, None,
                                    None, 0, None) == bad
    assert lib.oscar_commit_draft(None, 0, 1, 4, None, None, None, None, 1, None, None, 0, None, None) == bad


def _rope(osc, N=1, dim=128, dtype=0, rot=128, layout=0, scale=1.0, inverse=0, heads=1, ptr=4096, strides=(128, 128),
          pos=4096, turns=4096, out=None):
    t = osc.RopeTensor(ptr, ptr if out is None else out, strides[0], strides[1], 128, 128, heads)
    none = osc.RopeTensor()
    return osc.lib().oscar_rope(ctypes.byref(t), ctypes.byref(none), N, dim, dtype, pos, turns, rot, layout, scale, inverse,
                                None)


@pytest.mark.parametrize("kw", [
    dict(N=-1), dict(dim=0), dict(rot=0), dict(rot=3), dict(rot=130), dict(dtype=3), dict(layout=2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(inverse=2), dict(heads=-1), dict(ptr=0), dict(ptr=4097),
    dict(strides=(-1, 128)), dict(pos=0), dict(turns=0), dict(strides=(256, 128)),   # in place with other strides
])
def test_rope_refusals(osc, kw):
    assert _rope(osc, **kw) == osc.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dim=129), dict(dim=514)])
def test_rope_unsupported(osc, kw):
    assert _rope(osc, **kw) == osc.ERR_UNSUPPORTED


def test_rope_of_nothing_is_fine(osc):
    assert _rope(osc, N=0, ptr=0) == 0 and _rope(osc, heads=0, ptr=0) == 0


def _freq(osc, rot, base, kind, factor=1.0, orig=0.0, fast=32.0, slow=1.0):
    f, s = np.full(max(1, rot // 2), np.nan), ctypes.c_float(-1)
    rc = osc.lib().oscar_rope_frequencies(rot, base, kind, factor, orig, fast, slow, f.ctypes.data, ctypes.byref(s))
    return rc, f, s.value


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (24, 1e6), (128, 1e6), (256, 5e5)])
def test_frequencies_follow_their_formulas(osc, rot, base):
    half = rot // 2
    f0 = base ** (-np.arange(half) / half)
    rc, f, s = _freq(osc, rot, base, osc.ROPE_NONE)
    assert rc == 0 and s == 1.0 and np.allclose(f, f0, rtol=1e-14)
    rc, f, s = _freq(osc, rot, base, osc.ROPE_LINEAR, 4.0)
    assert rc == 0 and s == 1.0 and np.allclose(f, f0 / 4, rtol=1e-14)
    if rot > 2:
        rc, f, s = _freq(osc, rot, base, osc.ROPE_NTK, 8.0)
        b = base * 8.0 ** (rot / (rot - 2))
        assert rc == 0 and np.allclose(f, b ** (-np.arange(half) / half), rtol=1e-13)
        assert np.isclose(f[-1], f0[-1] / 8.0, rtol=1e-12)   # the slowest pair is stretched by the factor
    rc, f, s = _freq(osc, rot, base, osc.ROPE_YARN, 4.0, 32768.0)
    assert rc == 0 and np.isclose(s, 0.1 * np.log(4.0) + 1, rtol=1e-6)
    turns = 32768.0 * f0 / (2 * np.pi)
    # pairs well inside a regime are wholly kept or wholly stretched; nothing leaves the two
    step = base ** (1 / half)
    assert np.allclose(f[turns > 32 * step * 1.01], f0[turns > 32 * step * 1.01], rtol=1e-14)
    assert np.allclose(f[turns < 1 / step / 1.01], f0[turns < 1 / step / 1.01] / 4, rtol=1e-14)
    assert np.all(f <= f0 * (1 + 1e-14)) and np.all(f >= f0 / 4 * (1 - 1e-14))


@pytest.mark.parametrize("args", [
    (0, 1e4, 0), (3, 1e4, 0), (64, 1.0, 0), (64, float("inf"), 0), (64, 1e4, 4), (64, 1e4, -1), (64, 1e4, 1, 0.5),
    (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096.0, 1.0, 2.0), (64, 1e4, 3, 2.0, 4096.0, 32.0, 0.0),
])
def test_frequency_refusals(osc, args):
    assert _freq(osc, *args)[0] == osc.ERR_INVALID_ARG


def test_turns_are_64_bit_fractions(osc):
    from fractions import Fraction
    pi = Fraction("3.14159265358979323846264338327950288419716939937510")
    f = np.array([1.0, 0.5, 1e-7, 0.0, 6.28])
    t = np.zeros(5, np.uint64)
    assert osc.lib().oscar_rope_turns(f.ctypes.data, 5, t.ctypes.data) == 0
    for x, y in zip(f, t):
        want = Fraction(float(x)) / (2 * pi) * 2 ** 64
        assert abs(int(y) - want) <= 1
    for bad in (-1e-9, 2 * np.pi, np.nan, np.inf):
        f[2] = bad
        assert osc.lib().oscar_rope_turns(f.ctypes.data, 5, t.ctypes.data) == osc.ERR_INVALID_ARG
    assert osc.lib().oscar_rope_turns(None, 5, t.ctypes.data) == osc.ERR_INVALID_ARG
    assert osc.lib().oscar_rope_turns(f.ctypes.data, 0, t.ctypes.data) == osc.ERR_INVALID_ARG
