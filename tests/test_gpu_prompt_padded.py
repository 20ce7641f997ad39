"""Prompt attention where most bounds are padding: empty prompts behind the last real one, up to the most that a call takes.
The call gives the results of the real prompts alone, and no bounded wait runs out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import prompt_cases as C  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

SM = 1.0 / 128 ** 0.5


def case(seed, n, hq, hkv):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, k, v = (torch.randn(n, h, 128, generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv))
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hq, num_int2_pages=1, num_bf16_pages=5))
    return cache, q, k, v


# (prompts, query heads, key heads): a server's batch, many, and 2^24 prompts times key heads
@pytest.mark.parametrize("B,hq,hkv", [(4096, 32, 8), (16_384, 8, 8), (131_072, 32, 8), (2 ** 21, 8, 8), (2 ** 24, 1, 1),
                                      (2 ** 18, 64, 64)])
def test_padding_behind_the_prompts(B, hq, hkv):
    lens = [140, 0, 61]
    cache, q, k, v = case(B % 97, sum(lens), hq, hkv)
    cu = torch.full((B + 1,), sum(lens), dtype=torch.int32, device=DEV)
    cu[:4] = torch.tensor([0, 140, 140, 201], device=DEV)
    lse = torch.zeros(sum(lens), hq, device=DEV)
    out = cache.prompt_attention(q, k, v, cu, SM, lse=lse)
    assert cache.get_status() == 0
    C.check(out, lse, q, k, v, lens, [0, 140, 140], SM)
    assert torch.equal(out, cache.prompt_attention(q, k, v, cu[:4].clone(), SM))


def test_a_captured_call_for_the_most_prompts():
    most, n = 4096, 700
    cache, q, k, v = case(5, n, 32, 8)
    cu, out = torch.zeros(most + 1, dtype=torch.int32, device=DEV), torch.zeros_like(q)
    cache.prompt_attention(q, k, v, cu, SM, out=out)                     # all of it padding
    assert cache.get_status() == 0 and (out == 0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.prompt_attention(q, k, v, cu, SM, out=out)
    for lens in ([700], [1, 699], [100] * 7, [0, 350, 0, 350], [7] * 100, []):
        real = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        cu.fill_(int(real[-1]))
        cu[:len(real)] = torch.as_tensor(real, device=DEV)
        out.zero_()
        graph.replay()
        assert cache.get_status() == 0
        want = torch.zeros_like(out)
        cache.prompt_attention(q, k, v, real, SM, out=want)
        assert torch.equal(out, want)
