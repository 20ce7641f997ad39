"""Causal attention of packed prompts on the GPU against 64-bit softmax attention (reference and bound: prompt_cases.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import prompt_cases as C  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

SM = 1.0 / 128 ** 0.5


def cache_of(hq, hkv):
    return osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hq, num_int2_pages=1, num_bf16_pages=5))


def rows(seed, n, hq, hkv):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, hq + 2 * hkv, 128, generator=g, device=DEV)
    x[:, hq + hkv:] += 0.5                                               # values with a mean
    x = x.bfloat16()
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]                 # views of one buffer


def bounds(lens, first=0):
    return (first + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)


LENS = [[1], [2], [31, 33], [63, 64, 65], [127, 128, 129], [191, 192, 193], [255, 256, 257], [0, 5, 0, 129, 1, 700, 0],
        [1] * 70, [385], [513, 3], [1025]]


@pytest.mark.parametrize("gq", [1, 2, 4, 8])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, gq):
    hkv = 2
    q, k, v = rows(len(lens) + gq, sum(lens), hkv * gq, hkv)
    cu, cache = bounds(lens), cache_of(hkv * gq, hkv)
    lse = torch.full((sum(lens), hkv * gq), 7.0, device=DEV)
    out = cache.prompt_attention(q, k, v, cu, SM, lse=lse)
    C.check(out, lse, q, k, v, lens, cu[:-1], SM)
    wide = cache.prompt_attention(q, k, v, cu, SM, out_dtype=osc.OUT_FP32)
    C.check(wide, None, q, k, v, lens, cu[:-1], SM)
    assert torch.equal(wide.bfloat16(), out) and cache.get_status() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (64, 8), (12, 12)])
def test_heads(hq, hkv):
    lens = [77, 300]
    q, k, v = rows(hq, sum(lens), hq, hkv)
    cu = bounds(lens)
    out = cache_of(hq, hkv).prompt_attention(q, k, v, cu, SM)
    C.check(out, None, q, k, v, lens, cu[:-1], SM)


@pytest.mark.parametrize("scale", [1e-30, 0.01, 1.0, 40.0, 1e6])
def test_scales(scale):
    q, k, v = rows(3, 400, 4, 2)
    cu = bounds([400])
    out = cache_of(4, 2).prompt_attention(q, k, v, cu, scale)
    assert out.isfinite().all()
    if scale <= 1.0:
        C.check(out, None, q, k, v, [400], [0], scale)
    else:                                                                # nearly one token's value: it is one of the largest logits'
        x = torch.einsum("qhd,khd->hqk", q.double(), k.double().repeat_interleave(2, 1))
        x = x.masked_fill(torch.ones(400, 400, dtype=torch.bool, device=DEV).triu(1), -torch.inf)
        top, at = x.topk(2, -1)
        sure = ((top[..., 0] - top[..., 1]) * scale > 40).T               # [q, h]
        want = v.repeat_interleave(2, 1).permute(1, 0, 2).gather(1, at[..., :1].expand(-1, -1, 128)).transpose(0, 1)
        # the weight of one token is at least 2^-10 and bf16: off by 2^-8 of itself against its float32 sum
        off = (out.double() - want.double()).abs()[sure]
        assert sure.float().mean() > 0.5 and (off <= 2.0 ** -6.9 * want.double().abs()[sure]).all()


@pytest.mark.parametrize("gq", [1, 4])
@pytest.mark.parametrize("kind", ["rising", "falling", "late", "equal"])
def test_maxima_that_move(kind, gq):
    # logits that rise or fall along the prompt by far more than 2^10 between blocks; one late token that outweighs all
    n = 900
    q, k, v = rows(9, n, 2 * gq, 2)
    q, k = q.clone(), k.clone()
    q[..., 0], k[..., 1:] = 8.0, k[..., 1:] * 0.1
    ramp = torch.linspace(0, 60, n, device=DEV)[:, None]
    k[..., 0] = {"rising": ramp, "falling": 60 - ramp, "late": (torch.arange(n, device=DEV) == 700)[:, None] * 50.0,
                 "equal": ramp * 0}[kind].bfloat16()
    cache, cu = cache_of(2 * gq, 2), bounds([n])
    lse = torch.zeros(n, 2 * gq, device=DEV)
    out = cache.prompt_attention(q, k, v, cu, SM, lse=lse)
    C.check(out, lse, q, k, v, [n], [0], SM)


def test_a_long_prompt():
    n = 20_011
    q, k, v = rows(5, n + 6, 8, 2)
    cu = bounds([n], first=4)
    want = set(np.random.default_rng(1).integers(4, n + 4, 60).tolist()) | {4, n + 3}
    lse = torch.zeros(n + 6, 8, device=DEV)
    out = cache_of(8, 2).prompt_attention(q, k, v, cu, SM, lse=lse)
    C.check(out, lse, q, k, v, [n], [4], SM, rows=want)


@pytest.mark.parametrize("gq", [1, 8])
def test_rows_of_no_prompt_stay_and_are_not_seen(gq):
    lens, first, tail = [200, 0, 61], 33, 90
    n = first + sum(lens) + tail
    q, k, v = (x.clone() for x in rows(6, n, 2 * gq, 2))
    for x in (q, k, v):
        x[:first], x[first + sum(lens):] = float("nan"), float("inf")
    cu, cache = bounds(lens, first), cache_of(2 * gq, 2)
    out, lse = torch.full_like(q, -3.0), torch.full((n, 2 * gq), -3.0, device=DEV)
    cache.prompt_attention(q, k, v, cu, SM, out=out, lse=lse)
    assert cache.get_status() == 0
    C.check(out, lse, q, k, v, lens, cu[:-1], SM)
    for x in (out, lse):
        assert (x[:first] == -3).all() and (x[first + sum(lens):] == -3).all()


@pytest.mark.parametrize("gq", [1, 2, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_non_finite_rows_reach_only_what_sees_them(which, bad, gq):
    lens = [150, 300]
    n, hkv = sum(lens), 2
    q, k, v = (x.clone() for x in rows(7, n, hkv * gq, hkv))
    cu, cache = bounds(lens), cache_of(hkv * gq, hkv)
    want = cache.prompt_attention(q, k, v, cu, SM)
    assert cache.get_status() == 0
    head = 1
    for at in (150 + 0, 150 + 63, 150 + 130, 150 + 299, 149):
        t = {"q": q, "k": k, "v": v}[which]
        keep = t[at, head].clone()
        t[at, head, 17] = bad
        out = cache.prompt_attention(q, k, v, cu, SM)
        # an infinite key's logit may be -inf, a weight of 0: then its rows are finite
        assert cache.get_status() == (0 if out.isfinite().all() else osc.STATUS_NONFINITE)
        end = 150 if at < 150 else 450
        hit = torch.zeros(n, hkv * gq, dtype=torch.bool, device=DEV)
        if which == "q":
            hit[at, head] = True
        else:
            hit[at:end, head * gq:(head + 1) * gq] = True
        assert torch.equal(out[~hit], want[~hit])
        if which == "v" or bad != bad:
            assert (~out[hit].isfinite()).any(-1).all()
        t[at, head] = keep


def test_bounds_out_of_order_stay_within_the_buffers():
    q, k, v = rows(8, 300, 4, 2)
    cache = cache_of(4, 2)
    for cu in ([0, 400], [-5, 100, 300], [0, 200, 100, 300], [500, 600], [2 ** 31 - 1, -2 ** 31]):
        cache.prompt_attention(q, k, v, np.array(cu, np.int32), SM)
        assert cache.get_status() == osc.STATUS_BAD_SEQLEN
    out = cache.prompt_attention(q, k, v, np.array([0, 400], np.int32), SM)     # the end is taken as 300
    assert torch.equal(out, cache.prompt_attention(q, k, v, np.array([0, 300], np.int32), SM))


def test_strides_streams_and_graphs():
    lens = [129, 64, 300]
    n = sum(lens)
    q, k, v = rows(10, n, 8, 2)
    cu, cache = torch.as_tensor(bounds(lens), device=DEV), cache_of(8, 2)
    want = cache.prompt_attention(q, k, v, cu, SM)
    flat = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)    # noqa: E731  heads outermost
    assert torch.equal(cache.prompt_attention(flat(q), flat(k), v.contiguous(), cu, SM), want)
    streams, outs = [torch.cuda.Stream() for _ in range(3)], [torch.zeros_like(want) for _ in range(3)]
    for s, o in zip(streams, outs):                                      # at once: nothing is shared
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            cache.prompt_attention(q, k, v, cu, SM, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        k2 = k * 1                                                       # from the kernel just before
        cache.prompt_attention(q, k2, v, cu, SM, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    cu.copy_(torch.as_tensor(bounds([0, n, 0]), device=DEV))             # other bounds in the same graph
    graph.replay()
    assert torch.equal(out, cache.prompt_attention(q, k, v, bounds([n]), SM))
    assert cache.get_status() == 0


def test_refusals_and_nothing_to_do():
    q, k, v = rows(11, 40, 8, 2)
    cache, cu = cache_of(8, 2), bounds([40])
    good = dict(q=q, k=k, v=v, cu_seqlens=cu, sm_scale=SM)
    odd = torch.zeros(40, 8 * 128 + 4, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(q=q.float()), dict(k=k[:39]), dict(v=q), dict(q=q[:, :4]), dict(sm_scale=0.0), dict(sm_scale=float("nan")),
                dict(out=torch.zeros(40, 8, 128, device=DEV)), dict(out_dtype=2), dict(lse=torch.zeros(40, 2, device=DEV)),
                dict(q=odd[:, 4:].unflatten(1, (8, 128))), dict(q=odd[:, :1024].unflatten(1, (8, 128))),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(cu_seqlens=np.zeros((2, 2), np.int32)),
                dict(k=k[:1].expand(40, 2, 128)), dict(cu_seqlens=np.zeros(0, np.int32))):
        with pytest.raises(osc.OscarError):
            cache.prompt_attention(**{**good, **bad})
    assert cache.prompt_attention(q[:0], k[:0], v[:0], np.zeros(1, np.int32), SM).shape == (0, 8, 128)
    out = torch.full_like(q, 5.0)
    cache.prompt_attention(q, k, v, np.zeros(1, np.int32), SM, out=out)  # no prompts
    cache.prompt_attention(q, k, v, np.zeros(9, np.int32), SM, out=out)  # empty ones
    assert (out == 5).all() and cache.get_status() == 0


@pytest.mark.parametrize("gq", [1, 4])
def test_many_items_for_a_cta(gq):
    # dozens of items a CTA, of all lengths; then values that are not finite in some prompts, between others that are
    hkv, B = 8, 400
    g = torch.Generator().manual_seed(gq)
    lens = torch.randint(0, 420, (B,), generator=g).tolist()
    n, cu = sum(lens), bounds(lens)
    q, k, v = (x.clone() for x in rows(12, n, hkv * gq, hkv))
    cache = cache_of(hkv * gq, hkv)
    lse = torch.zeros(n, hkv * gq, device=DEV)
    out = cache.prompt_attention(q, k, v, cu, SM, lse=lse)
    some = set(torch.randint(0, n, (80,), generator=g).tolist())
    C.check(out, lse, q, k, v, lens, cu[:-1], SM, rows=some)
    for _ in range(3):                                                   # whoever takes what: the same bits
        assert torch.equal(cache.prompt_attention(q, k, v, cu, SM), out)
    hit = torch.zeros(n, hkv * gq, dtype=torch.bool, device=DEV)
    for r in range(0, B, 3):
        if lens[r] == 0:
            continue
        at, h = int(cu[r]) + (7 * r) % lens[r], r % hkv
        v[at, h, r % 128] = (float("nan"), float("inf"), -float("inf"))[r // 3 % 3]
        hit[at:int(cu[r + 1]), h * gq:(h + 1) * gq] = True
    got = cache.prompt_attention(q, k, v, cu, SM)
    assert cache.get_status() == osc.STATUS_NONFINITE
    assert torch.equal(got[~hit], out[~hit]) and (~got[hit].isfinite()).any(-1).all()


def test_more_prompts_than_a_search_holds():
    # thousands of prompts, most of them empty, the others where searches of 32 begin and end
    lens = [0] * 5000
    for i, at in enumerate((0, 31, 32, 33, 1023, 1024, 2047, 3000, 4095, 4990, 4999)):
        lens[at] = 1 + 37 * i
    q, k, v = rows(13, sum(lens), 8, 2)
    cu, cache = bounds(lens), cache_of(8, 2)
    out = cache.prompt_attention(q, k, v, cu, SM)
    C.check(out, None, q, k, v, lens, cu[:-1], SM)
    assert cache.get_status() == 0


def test_more_prompts_than_a_call_takes():
    # the most prompts (times key heads) that a call takes, all but four of them empty, and one more
    q, k, v = rows(14, 300, 64, 64)
    cache, most = cache_of(64, 64), 2 ** 24 // 64
    cu = torch.zeros(most + 2, dtype=torch.int32, device=DEV)
    cu[7:], cu[40_000:], cu[200_000:], cu[most:] = 1, 130, 131, 300
    out = cache.prompt_attention(q, k, v, cu[:-1], SM)
    lens = [1, 129, 1, 169]
    C.check(out, None, q, k, v, lens, [0, 1, 130, 131], SM)
    assert cache.get_status() == 0
    with pytest.raises(osc.OscarError):
        cache.prompt_attention(q, k, v, cu, SM)
