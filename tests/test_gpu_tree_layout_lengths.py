"""Lengths that oscar_tree_layout cannot place nodes behind."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


@pytest.mark.parametrize("T", [1, 5, 70])
def test_lengths_out_of_range(T):
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=1, num_bf16_pages=5,
                                           max_batch=1, max_splits=1), device=DEV)
    parents = np.tile(np.arange(T) - 1, (2, 1))
    top = 2 ** 31 - 1 - T
    mask, pos = cache.tree_layout(parents, [0, top])
    assert cache.get_status() == 0
    assert pos.tolist() == [list(range(T)), list(range(top, top + T))]
    for bad in (-1, -2 ** 31, top + 1, 2 ** 31 - 1):
        m, p = cache.tree_layout(parents, [0, bad])
        assert cache.get_status() == osc.STATUS_BAD_SEQLEN
        assert torch.equal(m[0], mask[0]) and torch.equal(p[0], pos[0])
        assert (m[1] == 0).all() and (p[1] == -1).all()


def test_a_padded_request_may_hold_any_length():
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=1, num_bf16_pages=5,
                                           max_batch=1, max_splits=1), device=DEV)
    mask, pos = cache.tree_layout([[-1, 0]] * 4, [7, -1, -2 ** 31, 2 ** 31 - 1], n_draft=[2, 0, 0, 0])
    assert cache.get_status() == 0
    assert pos.tolist() == [[7, 8]] + [[-1, -1]] * 3 and mask.flatten().tolist() == [1, 3] + [0] * 6
