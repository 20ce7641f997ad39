"""Values, keys and queries of prompts that are not finite: what reaches which channel of which row, and its lse. A value does
the same wherever it lies: in the tokens that all rows of a tile see, in those that only some see, in its first or last
group. The weights are at least 2^-60 here, so that a value of infinity is one in the result; all else has the bits of the
call with finite inputs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

SM = 1.0 / 128 ** 0.5
NAN, INF = float("nan"), float("inf")
LENS = [150, 700, 1]


def case(seed, gq, hkv=2, lens=LENS):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, hq = sum(lens), gq * hkv
    x = torch.randn(n, hq + 2 * hkv, 128, generator=g, device=DEV).bfloat16()
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hq, num_int2_pages=1, num_bf16_pages=5))
    cu = torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device=DEV)
    return cache, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], cu


def call(cache, q, k, v, cu, dtype):
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    return cache.prompt_attention(q, k, v, cu, SM, out_dtype=dtype, lse=lse), lse


def same(a, b):
    """Equal bits, or NaN in both places."""
    return ((a == b) | (a.isnan() & b.isnan())).all()


@pytest.mark.parametrize("gq", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", [0, 1])
def test_a_value_reaches_its_channel(gq, dtype):
    cache, q, k, v, cu = case(1, gq)
    want, want_lse = call(cache, q, k, v, cu, dtype)
    assert cache.get_status() == 0
    head, rows = 1, slice(gq, 2 * gq)
    for i, at in enumerate([0, 149, 150, 151, 150 + 63, 150 + 64, 150 + 127, 150 + 130, 150 + 255, 150 + 256, 150 + 400, 150 + 640,
                            150 + 699, 850]):
        end = 150 if at < 150 else 850 if at < 850 else 851
        channel, bad = (17 + 37 * i) % 128, (NAN, INF, -INF)[i % 3]
        v2 = v.clone()
        v2[at, head, channel] = bad
        expected = want.clone()
        expected[at:end, rows, channel] = bad
        out, lse = call(cache, q, k, v2, cu, dtype)
        assert cache.get_status() == osc.STATUS_NONFINITE
        assert same(out, expected) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("gq", [1, 4])
@pytest.mark.parametrize("dtype", [0, 1])
def test_several_values(gq, dtype):
    cache, q, k, v, cu = case(2, gq)
    v = v.transpose(0, 1).contiguous().transpose(0, 1)                   # heads outermost
    want, want_lse = call(cache, q, k, v, cu, dtype)
    bad = [(150 + 300, 3, INF), (150 + 310, 3, -INF), (150 + 500, 90, INF), (150 + 690, 90, INF), (150 + 690, 91, NAN),
           (150 + 695, 127, -INF), (20, 0, -INF), (149, 64, INF)]
    expected = want.clone()
    for at, channel, x in bad:
        v[at, 0, channel] = x
        expected[at:150 if at < 150 else 850, :gq, channel] += x         # INF and -INF: NaN
    v[150 + 698, 1] = INF                                                # a whole row
    expected[150 + 698:850, gq:] = INF
    out, lse = call(cache, q, k, v, cu, dtype)
    assert cache.get_status() == osc.STATUS_NONFINITE
    assert same(out, expected) and torch.equal(lse, want_lse)


def check_hit(out, lse, hit, x):
    """The hit rows [n]: by the logits that are not finite, x [n, keys] (0 for the finite ones, the keys that the row sees)."""
    nan, none = (x.isnan() | (x == INF)).any(-1), (x == -INF).all(-1)    # no weights at all: 0 / 0, and the log of 0
    out, lse = out[hit], lse[hit]
    assert out[nan].isnan().all() and lse[nan].isnan().all()
    assert out[none].isnan().all() and (lse[none] == -INF).all()
    assert out[~nan & ~none].isfinite().all() and lse[~nan & ~none].isfinite().all()


@pytest.mark.parametrize("gq", [1, 8])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_queries_and_keys(gq, bad):
    cache, q, k, v, cu = case(3, gq)
    want, want_lse = call(cache, q, k, v, cu, 0)
    assert cache.get_status() == 0
    for at in (3, 150, 150 + 200, 150 + 699):
        start, end = (0, 150) if at < 150 else (150, 850)
        q2 = q.clone()
        q2[at, gq, 5] = bad
        out, lse = call(cache, q2, k, v, cu, 0)
        hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
        hit[at, gq] = True
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
        check_hit(out, lse, hit, (bad * k[start:at + 1, 1, 5].double())[None])
        assert cache.get_status() == (0 if out.isfinite().all() else osc.STATUS_NONFINITE)
        k2 = k.clone()
        k2[at, 1, 5] = bad
        out, lse = call(cache, q, k2, v, cu, 0)
        hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
        hit[at:end, gq:] = True
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
        x = torch.zeros(end - at, gq, 2, device=DEV, dtype=torch.float64)
        x[..., 0] = bad * q[at:end, gq:, 5].double()
        if at == start:
            x[0, :, 1] = -INF                                            # its own row sees no other key
        check_hit(out, lse, hit, x.reshape(-1, 2))
        assert cache.get_status() == (0 if out.isfinite().all() else osc.STATUS_NONFINITE)
