"""What appends and steps from raw projections report, and what they leave alone: rows that become infinite in the rounding to
bf16, lengths below 0 and pages out of range."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    import gpu_cases as G
    DEV = torch.device("cuda:0")

SM = 1.0 / 128 ** 0.5
MOST = torch.finfo(torch.bfloat16).max                                   # 3.3895e38; 3.3961e38 and more round to infinity


def case(lens, hkv, gq, seed, **kw):
    cache, _, hist, bf = G.build_decode_case([n + 1 for n in lens], hkv, gq, 0, seed, **kw)
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, k, v = (torch.randn(len(lens), h, 128, generator=g, device=DEV).bfloat16() for h in (hkv * gq, hkv, hkv))
    return cache, q, k, v, torch.as_tensor(hist, device=DEV), torch.as_tensor(bf, device=DEV)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("which", ["q", "k"])
def test_rows_that_round_to_infinity(which, step):
    lens = [100, 400]
    cache, q, k, v, hist, bf = case(lens, 2, 4, 21, algo=1)
    sl, pos = np.array(lens, np.int32), np.zeros(2, np.int32)            # at position 0: the scale alone
    call = (lambda p: cache.decode_step_rope(0, p, q, k, v, sl, hist, bf, SM, eps=None, positions=pos, q_out=out)) if step \
        else (lambda p: cache.append_kv_rope(0, p, q, k, v, sl, hist, bf, eps=None, positions=pos, q_out=out))
    x, out = (q if which == "q" else k), torch.zeros_like(q)
    x[1, 1, 7], x[1, 1, 71] = MOST, 0.0                                  # the pair (7, 71)
    call(osc.RopePlan(128, scale=0.5))
    assert cache.get_status() == 0
    call(osc.RopePlan(128, scale=1.003))                                 # 3.3997e38: float32 holds it, bf16 does not
    assert cache.get_status() == osc.STATUS_NONFINITE
    assert which == "k" or (out[1, 1, 7] == float("inf") and out.isinf().sum() == 1)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("normed", [True, False])
def test_a_refused_request_leaves_the_pool_alone(step, normed):
    lens = [700, 30, 400]
    cache, q, k, v, hist, bf = case(lens, 2, 4, 22, algo=1)
    plan, eps = osc.RopePlan(128), 1e-6 if normed else None
    bad_page = bf.clone()
    bad_page[0] = 10 ** 6                                                # every page of the first request
    bad_hist = hist.clone()
    bad_hist[0] = -5
    before = cache.pool.clone()
    for change, status in ((dict(sl=[-1, 30, 400]), osc.STATUS_BAD_SEQLEN), (dict(sl=[-2 ** 31, 30, 400]), osc.STATUS_BAD_SEQLEN),
                           (dict(bf=bad_page), osc.STATUS_BAD_PAGE), (dict(bf=bad_page, hist=bad_hist), osc.STATUS_BAD_PAGE)):
        cache.pool.copy_(before)
        a = dict(sl=lens, bf=bf, hist=hist) | change
        sl = torch.tensor(a["sl"], dtype=torch.int32, device=DEV)
        if step:
            cache.decode_step_rope(0, plan, q, k, v, sl, a["hist"], a["bf"], SM, eps=eps)
        else:
            cache.append_kv_rope(0, plan, q, k, v, sl, a["hist"], a["bf"], eps=eps)
        assert cache.get_status() & status
        # what the other requests write is known from a call without the first
        got = cache.pool.clone()
        cache.pool.copy_(before)
        good = (plan, q[1:], k[1:], v[1:], sl[1:].clone(), hist[1:].clone(), bf[1:].clone())
        cache.append_kv_rope(0, *good, eps=eps)
        assert cache.get_status() == 0
        assert torch.equal(got, cache.pool) and not torch.equal(got, before)
