"""CPU checks of the numbers of heads that the rotary calls take."""
import pytest


@pytest.fixture(scope="module")
def osc():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_decode_gb300 as o
    return o


def _row(osc, heads):
    return osc.RopeTensor(4096, 4096, 128, 128, 128, 128, heads)


@pytest.mark.parametrize("hq,hkv", [(2 ** 30 + 1, 0), (2 ** 30, 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_more_heads_than_rows_are_counted_in(osc, hq, hkv):
    lib, q, k = osc.lib(), _row(osc, hq), _row(osc, hkv)
    rotary = osc.Rotary(4096, 0, 1, 128, 0, 1.0)
    assert lib.oscar_rope(q, k, 1, 128, 0, 4096, 4096, 128, 0, 1.0, 0, None) == osc.ERR_UNSUPPORTED
    assert lib.oscar_rope_axes(q, k, 1, 128, 0, 4096, rotary, 0, None) == osc.ERR_UNSUPPORTED
    assert lib.oscar_rope_axes(q, k, 0, 128, 0, 4096, rotary, 0, None) == osc.ERR_UNSUPPORTED
