"""Pointers that are off their type's boundary are refused on the host."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def osc():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_decode_gb300 as o
    return o


@pytest.mark.parametrize("off", [1, 4])
def test_rope_turns(osc, off):
    t, none = osc.RopeTensor(4096, 4096, 128, 128, 128, 128, 1), osc.RopeTensor()
    rc = osc.lib().oscar_rope(ctypes.byref(t), ctypes.byref(none), 1, 128, 0, 4096, 4096 + off, 128, 0, 1.0, 0, None)
    assert rc == osc.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("off", [1, 4])
def test_masks(osc, off):
    torch = pytest.importorskip("torch")
    c = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=1, num_bf16_pages=5,
                                       max_batch=1, max_splits=1))
    x = torch.zeros(4096, dtype=torch.int64, device="cuda").data_ptr()
    lib = osc.lib()
    assert lib.oscar_tree_layout(c._h, 1, 2, x, None, x, x + 512 + off, x, None) == osc.ERR_INVALID_ARG
    ws = torch.empty(c.tree_workspace_bytes(1, 2, 1), dtype=torch.uint8, device="cuda")
    rc = lib.oscar_tree_attention(c._h, 0, 1, 2, x, x, x, x + off, None, x, x, 1, x, 0.1, x, 0, None, ws.data_ptr(), ws.numel(), None)
    assert rc == osc.ERR_INVALID_ARG
    assert c.get_status() == 0
