"""A call straight after the bulk prefill sees all of it: the sink and recent rows too, which a kernel of their own copies
beside the history's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


@pytest.mark.parametrize("L", [320, 330])                  # no history, and one page of ten rows
@pytest.mark.parametrize("what", ["tree", "decode"])
def test_attention_straight_after_the_prefill(L, what):
    B, hkv, gq = 512, 8, 1                                 # 1.3 GB of BF16 rows: the copy outlasts the history kernel
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hkv * gq, num_int2_pages=B,
                                           num_bf16_pages=5 * B, max_batch=B, max_splits=1), device=DEV)
    eye, tau = np.tile(np.eye(128, dtype=np.float32), (hkv, 1, 1)), np.full((hkv, 128), 4, np.float32)
    cache.set_rotation(0, eye, eye, tau, tau)
    g = torch.Generator(device=DEV).manual_seed(L)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)   # noqa: E731
    cu, lens = i32(np.arange(B + 1) * L), i32([L] * B)
    hist, bf = i32(np.arange(B)[:, None]), i32(np.arange(5 * B).reshape(B, 5))
    q = torch.randn(B, 1, hkv * gq, 128, generator=g, device=DEV).bfloat16()
    kd = torch.randn(B, 1, hkv, 128, generator=g, device=DEV).bfloat16()
    mask = torch.ones(B, 1, 1, dtype=torch.int64, device=DEV)
    ws = torch.empty(cache.tree_workspace_bytes(B, 1, 1), dtype=torch.uint8, device=DEV)

    def attend():
        if what == "tree":
            return cache.tree_attention(0, q, kd, kd, mask, lens, hist, bf, 0.1, workspace=ws)
        return cache.decode_attention(0, q[:, 0], lens, hist, bf, 0.1)

    for _ in range(5):
        k, v = (torch.randn(B * L, hkv, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
        torch.cuda.synchronize()
        cache.quantize_prefill(0, k, v, cu, hist, bf)
        out = attend()
        torch.cuda.synchronize()
        assert torch.equal(out, attend())
    assert cache.get_status() == 0
