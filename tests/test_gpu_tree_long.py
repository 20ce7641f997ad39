"""Tree attention over many pages of one request and kv head: the sums stay exact to float32.

With q = 0 every token weighs the same, so a row's output is the plain mean of the values and any bias of the
accumulators shows in it. The values have one sign, and the reference rounds them as the kernel does (code scale + zero
once, to fp16): weights and products are exact, and only the tensor cores' sums are not. An accumulator takes at most 1,024 products and each may lose
one unit of its last place, 2^-23 of a sum that is never larger than the last one: 2^-13 in all. Joins and the merge
add some units of 2^-23 more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

D, P = 128, 64


def history(pages, seed):
    """INT2 page blocks [pages, 1, 5120] of values near 3, and the sum of their V over all tokens (float64 [128])."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    blk = torch.randint(0, 256, (pages, 5120), generator=g, device=DEV, dtype=torch.uint8)
    meta = torch.empty(pages, 2, P, 2, 2, device=DEV, dtype=torch.float16)          # K, V; row; group; scale, zero
    meta[..., 0] = 0.1 + 0.5 * torch.rand(meta.shape[:-1], generator=g, device=DEV)
    meta[..., 1] = 3 + 0.1 * torch.randn(meta.shape[:-1], generator=g, device=DEV)
    blk[:, 4096:] = meta.reshape(pages, -1).view(torch.uint8)
    t, c = torch.arange(P, device=DEV), torch.arange(D, device=DEV)
    words = blk[:, 2048:4096].contiguous().view(torch.int32).reshape(pages, D, 4)[:, c ^ ((c >> 4) & 7)]
    codes = (words[:, :, (t >> 1) & 3] >> (16 * (t & 1) + 4 * (t >> 4) + 2 * ((t >> 3) & 1))) & 3      # [pages, D, P]
    scale, zero = (meta[:, 1, :, :, k].double().transpose(1, 2).repeat_interleave(D // 2, 1) for k in range(2))
    return blk[:, None], (codes * scale + zero).half().double().sum((0, 2))


def mean_error(B, T, hq, pages, sink, recent, seed=1):
    nbf = (sink + recent) // P
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=hq, num_int2_pages=max(1, pages),
                                           num_bf16_pages=nbf, max_batch=B, max_splits=1, sink=sink, recent=recent), device=DEV)
    eye, tau = np.eye(D, dtype=np.float32)[None], np.full((1, D), 8, np.float32)
    cache.set_rotation(0, eye, eye, tau, tau)
    total = torch.zeros(D, dtype=torch.float64, device=DEV)
    if pages:
        blk, total = history(pages, seed)
        cache.int2_pages(0).copy_(blk.reshape(cache.int2_pages(0).shape))
    bf = cache.bf16_pages(0).view(torch.bfloat16).reshape(nbf, 2, P, D)
    g = torch.Generator(device=DEV).manual_seed(seed)
    bf.copy_(3 + 0.3 * torch.randn(bf.shape, generator=g, device=DEV))
    want = (total + bf[:, 1].double().sum((0, 1))) / (pages * P + sink + recent)
    lens = torch.full((B,), sink + recent + pages * P, dtype=torch.int32, device=DEV)
    hist = torch.arange(pages, device=DEV, dtype=torch.int32).repeat(B, 1)           # the same pages for all
    bp = torch.arange(nbf, device=DEV, dtype=torch.int32).repeat(B, 1)
    q = torch.zeros(B, T, hq, D, device=DEV, dtype=torch.bfloat16)
    kv = torch.zeros(B, T, 1, D, device=DEV, dtype=torch.bfloat16)
    lse = torch.empty(B, T, hq, device=DEV)
    out = cache.tree_attention(0, q, kv, kv, torch.zeros(B, T, -(-T // 64), dtype=torch.int64, device=DEV), lens, hist, bp, 0.1,
                               out_dtype=osc.OUT_FP32, lse=lse)
    assert cache.get_status() == 0
    assert (lse - np.log(lens[0].item())).abs().max() <= 2.0 ** -18
    return ((out.double() - want) / want).abs().max().item()


# batches that fill the GPU several times over, so that few slots a request would do for the time
@pytest.mark.parametrize("B,T,hq,pages", [(608, 1, 8, 8192), (160, 17, 8, 8192), (1, 1, 1, 5000)])
def test_long_histories(B, T, hq, pages):
    assert mean_error(B, T, hq, pages, 64, 256) <= 2.0 ** -13 + 2.0 ** -20


@pytest.mark.parametrize("B,T,hq", [(608, 1, 8), (304, 17, 8)])
def test_long_windows(B, T, hq):
    assert mean_error(B, T, hq, 0, 64, 64 * 2039) <= 2.0 ** -13 + 2.0 ** -20   # the longest window there is
