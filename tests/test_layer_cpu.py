"""CPU checks of the calls around the cache in a layer: refusals that need no device."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def osc():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_decode_gb300 as o
    return o


def _row(osc, heads=1, ptr=4096, strides=(128, 128), out=None):
    return osc.RopeTensor(ptr, ptr if out is None else out, strides[0], strides[1], 128, 128, heads)


def _rotary(osc, rot=128, layout=0, scale=1.0, axes=0, num_axes=1, turns=4096):
    return osc.Rotary(turns, axes, num_axes, rot, layout, scale)


BAD_ROWS = [dict(heads=-1), dict(ptr=0), dict(ptr=4097), dict(strides=(-1, 128)), dict(strides=(256, 128))]
BAD_ROTARY = [dict(rot=0), dict(rot=3), dict(rot=130), dict(layout=2), dict(scale=float("nan")), dict(num_axes=0),
              dict(num_axes=5), dict(turns=0), dict(turns=4097)]
BAD_CALL = [dict(N=-1), dict(dim=0), dict(dtype=3), dict(pos=0)]


def _split(kw, *groups):
    out = []
    for g in groups:
        names = {n for d in g for n in d}
        out.append({n: v for n, v in kw.items() if n in names})
    return out


def _axes(osc, kw):
    row, rot, call = _split(kw, BAD_ROWS, BAD_ROTARY, BAD_CALL + [dict(inverse=0)])
    call = dict(N=1, dim=128, dtype=0, pos=4096, inverse=0) | call
    return osc.lib().oscar_rope_axes(_row(osc, **row), osc.RopeTensor(), call["N"], call["dim"], call["dtype"], call["pos"],
                                     _rotary(osc, **rot), call["inverse"], None)


def _norm(osc, kw):
    row, rot, call = _split(kw, BAD_ROWS, BAD_ROTARY, BAD_CALL + [dict(eps=0, w=0)])
    call = dict(N=1, dim=128, dtype=0, pos=4096, eps=1e-6, w=4096) | call
    return osc.lib().oscar_norm_rope(_row(osc, **row), osc.RopeTensor(), call["N"], call["dim"], call["dtype"], call["pos"],
                                     _rotary(osc, **rot), osc.HeadNorm(call["w"], 0, call["eps"]), None)


def _grad(osc, kw):
    row, rot, call = _split(kw, BAD_ROWS, BAD_ROTARY, BAD_CALL + [dict(eps=0, w=0, dw=0, ws=0, size=0, g=0, gheads=0)])
    call = dict(N=1, dim=128, dtype=0, pos=4096, eps=1e-6, w=4096, dw=4096, ws=4096, size=1 << 30, g=8192, gheads=1) | call
    g = osc.RopeTensor(call["g"], 0, 128, 128, 0, 0, call["gheads"])
    return osc.lib().oscar_norm_rope_backward(_row(osc, **row), osc.RopeTensor(), g, osc.RopeTensor(), call["N"],
                                              call["dim"], call["dtype"], call["pos"], _rotary(osc, **rot),
                                              osc.HeadNorm(call["w"], 0, call["eps"]), call["dw"], 0, call["ws"],
                                              call["size"], None)


@pytest.mark.parametrize("kw", BAD_ROWS + BAD_ROTARY + BAD_CALL + [dict(inverse=2)])
def test_rope_axes_refusals(osc, kw):
    assert _axes(osc, kw) == osc.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_ROWS + BAD_ROTARY + BAD_CALL + [dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")),
                                                                   dict(eps=float("nan")), dict(w=4097)])
def test_norm_rope_refusals(osc, kw):
    assert _norm(osc, kw) == osc.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_ROWS + BAD_ROTARY + BAD_CALL + [
    dict(eps=0.0), dict(w=4097), dict(dw=4098), dict(ws=0), dict(ws=4100), dict(size=100), dict(g=0), dict(g=8193),
    dict(gheads=2), dict(gheads=0), dict(out=8192, ptr=4096, strides=(256, 256), g=8192)])
def test_norm_rope_backward_refusals(osc, kw):
    if "out" in kw:                                    # in the gradient's place with other strides
        row = osc.RopeTensor(4096, 8192, 128, 128, 256, 128, 1)
        g = osc.RopeTensor(8192, 0, 128, 128, 0, 0, 1)
        rc = osc.lib().oscar_norm_rope_backward(row, osc.RopeTensor(), g, osc.RopeTensor(), 1, 128, 0, 4096, _rotary(osc),
                                                osc.HeadNorm(0, 0, 1e-6), 0, 0, 0, 0, None)
    else:
        rc = _grad(osc, kw)
    assert rc == osc.ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_axes, _norm, _grad])
@pytest.mark.parametrize("dim", [129, 514])
def test_unsupported_heads(osc, call, dim):
    assert call(osc, dict(dim=dim)) == osc.ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [_norm, _grad])
def test_too_many_heads(osc, call):
    assert call(osc, dict(heads=8193, gheads=8193)) == osc.ERR_UNSUPPORTED


def test_missing_structures_and_no_work(osc):
    lib, none = osc.lib(), osc.RopeTensor()
    assert lib.oscar_rope_axes(_row(osc), none, 1, 128, 0, 4096, None, 0, None) == osc.ERR_INVALID_ARG
    assert lib.oscar_norm_rope(_row(osc), none, 1, 128, 0, 4096, _rotary(osc), None, None) == osc.ERR_INVALID_ARG
    for kw in (dict(N=0, ptr=0), dict(heads=0)):
        assert _axes(osc, kw) == 0 and _norm(osc, kw) == 0


def test_workspace_size(osc):
    n = ctypes.c_size_t()
    size = osc.lib().oscar_norm_rope_workspace_bytes
    assert size(128, ctypes.byref(n)) == 0 and n.value % 512 == 0 and n.value == osc.norm_rope_workspace_bytes(128)
    assert size(128, None) == size(0, ctypes.byref(n)) == osc.ERR_INVALID_ARG
    assert size(130 + 1, ctypes.byref(n)) == size(514, ctypes.byref(n)) == osc.ERR_UNSUPPORTED


@pytest.mark.parametrize("axes", [[0] * 31, [0] * 33, [-1] + [0] * 31, [4] + [0] * 31, [0.0] * 32])
def test_plan_refuses_bad_axes(osc, axes):
    with pytest.raises(osc.OscarError):
        osc.RopePlan(64, axes=axes, device="cpu")


def test_plan_with_axes(osc):
    p = osc.RopePlan(64, axes=np.repeat([0, 2], [10, 22]), device="cpu")
    assert p.num_axes == 3 and p.rotary(0).num_axes == 3 and p.axes.tolist() == [0] * 10 + [2] * 22
    assert osc.RopePlan(64, device="cpu").axes is None


def test_raw_steps_without_a_cache_are_refused(osc):
    lib, bad = osc.lib(), osc.ERR_INVALID_ARG
    assert lib.oscar_append_kv_rope(None, 0, 1, osc.RawStep(), None, None, 0, None, None) == bad
    assert lib.oscar_decode_step_rope(None, 0, 1, osc.RawStep(), None, None, 0, 0, None, 0.1, None, 0, None, None) == bad


def test_prompt_attention_without_a_cache_is_refused(osc):
    x = osc.Heads(4096, 128, 128)
    assert osc.lib().oscar_prompt_attention(None, 1, x, x, x, 4096, 1, 0.1, 4096, 0, None, None) == osc.ERR_INVALID_ARG
