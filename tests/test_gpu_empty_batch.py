"""The drafted-token calls with no request: nothing is launched, nothing is written, and the tensors returned are empty."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 8), (26, 32, 8), (256, 8, 1)])
@pytest.mark.parametrize("pages", [0, 1, 5000])
def test_no_requests(T, hq, hkv, pages):
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hq, num_int2_pages=2, num_bf16_pages=5,
                                           max_batch=1, max_splits=1), device=DEV)
    before = cache.pool.clone()
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)   # noqa: E731
    assert cache.tree_workspace_bytes(0, T, pages) >= 0
    mask, pos = cache.tree_layout(i32(0, T), i32(0))
    assert mask.shape == (0, T, (T + 63) // 64) and pos.shape == (0, T)
    q, k = (torch.zeros(0, T, h, 128, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv))
    qr, kr = osc.rope(osc.RopePlan(128), q.view(0, hq, 128), k.view(0, hkv, 128), pos.view(-1))
    assert qr.shape == (0, hq, 128) and kr.shape == (0, hkv, 128)
    for ws in (None, torch.empty(256, dtype=torch.uint8, device=DEV)):
        out = cache.tree_attention(0, q, k, k, mask, i32(0), i32(0, pages), i32(0, 5), 0.1, workspace=ws)
        assert out.shape == q.shape
    cache.commit_draft(0, k, k, i32(0), i32(0), i32(0, pages), i32(0, 5))
    free, rings = i32(2), torch.tensor([1, 2, 3, 2], dtype=torch.int32, device=DEV)
    _, cu, _ = cache.build_tables(i32(0), i32(0), i32(0, pages), i32(0, 5), free, i32(5), rings)
    assert cu.tolist() == [0] and rings.tolist() == [1, 2, 3, 2]
    assert cache.get_status() == 0 and torch.equal(cache.pool, before)


@pytest.mark.parametrize("most", [1, 3, 256])
def test_no_requests_with_paths(most):
    # more accepted nodes than T are allowed with a path; a path of no requests is a null pointer
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=2, num_bf16_pages=5,
                                           max_batch=1, max_splits=1), device=DEV)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)   # noqa: E731
    k = torch.zeros(0, 2, 1, 128, dtype=torch.bfloat16, device=DEV)
    cache.commit_draft(0, k, k, i32(0), i32(0), i32(0, 4), i32(0, 5), path=i32(0, most))
    with pytest.raises(osc.OscarError):
        cache.commit_draft(0, k, k, i32(0), i32(0), i32(0, 4), i32(0, 5), path=i32(0, 257))
    assert cache.get_status() == 0
