"""Tree attention with queries that are not finite, beside rows whose largest logits come late."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    from gpu_cases import DEV, build_decode_case, to_dev_bf16, tokens
    from test_gpu_tree import compare, dev, draft
import synth
from tree_cases import mask_words, random_mask

PAGES = 24


def late_queries(T, hkv, gq, L):
    """Every row's logits grow along the history: its query follows one token per page, each page's more than the
    one before, so that a page's largest weight is far more than 2^9 times the first page's."""
    q, kd, vd = draft(71, 1, T, hkv, gq)
    k, _ = tokens(71, 0, hkv, L, extra=1)
    for i in range(T):
        for h in range(hkv):
            for e in range(gq):
                c = 1.5 * (1 + (i + e) % 5)
                late = k[64 + 64 * (PAGES - 1 - (i % 8)) + 7 * e + 3, h]
                q[0, i, h * gq + e] = synth.bf16_round(0.02 * c * late)
    return q, kd, vd


@pytest.mark.parametrize("T", [24, 40])                    # rows of one tile and of two
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 3.3e38])
def test_a_bad_query_reaches_no_other_row(T, value):
    lens, hkv, gq = [64 + 256 + 64 * PAGES + 5], 2, 4
    case = build_decode_case(lens, hkv, gq, 0, seed=71)
    cache, _, hp, bp = case
    q, kd, vd = late_queries(T, hkv, gq, lens[0])
    mask = random_mask(np.random.default_rng(5), 1, T, "tree")
    words, sm = torch.from_numpy(mask_words(mask)).to(DEV), synth.sm_scale()

    def run(x):
        lse = torch.zeros(1, T, hkv * gq, device=DEV)
        out = cache.tree_attention(0, x, to_dev_bf16(kd), to_dev_bf16(vd), words, dev(lens), hp, bp, sm,
                                   out_dtype=osc.OUT_FP32, lse=lse)
        return out, lse

    clean, clean_lse = run(to_dev_bf16(q))
    assert cache.get_status() == 0
    compare(clean, clean_lse, case, lens, q, kd, vd, mask, [T], 0, sm)
    bad = to_dev_bf16(q)
    hurt = torch.zeros(1, T, hkv * gq, dtype=torch.bool, device=DEV)
    for i, e in ((1, 0), (7, 2), (T - 1, 5)):              # rows of several warps, of both kv heads
        hurt[0, i, e] = True
        if value > 1e38 and np.isfinite(value):            # finite, but its rotation overflows
            bad[0, i, e] = value
        else:
            bad[0, i, e, 40] = value
    out, lse = run(bad)
    assert cache.get_status() == (0 if np.isfinite(value) else osc.STATUS_NONFINITE)
    assert torch.equal(out[~hurt], clean[~hurt]) and torch.equal(lse[~hurt], clean_lse[~hurt])
    if not np.isfinite(value):
        assert out[hurt].isnan().all() and lse[hurt].isnan().all()


@pytest.mark.parametrize("L", [0, 90])
def test_a_bad_query_without_history(L):
    T, hkv, gq = 6, 1, 4
    case = build_decode_case([max(L, 1)], hkv, gq, 0, seed=72)
    cache, _, hp, bp = case
    q, kd, vd = (to_dev_bf16(x) for x in draft(72, 1, T, hkv, gq))
    mask = np.zeros((1, T, T), bool)
    mask[0, 1:, 0] = True                                  # node 0 sees no drafted node
    kd[0, 0, 0, 9] = 2.0
    q[0, :, 1, 9] = -np.inf                                # every logit of a row that sees node 0 alone is -inf
    q[0, :, 2, 9] = np.nan
    lse = torch.zeros(1, T, gq, device=DEV)
    out = cache.tree_attention(0, q, kd, vd, torch.from_numpy(mask_words(mask)).to(DEV), dev([L]), hp, bp, synth.sm_scale(),
                               out_dtype=osc.OUT_FP32, lse=lse)
    assert cache.get_status() == osc.STATUS_NONFINITE
    sees = torch.arange(T, device=DEV) > 0 if L == 0 else torch.ones(T, dtype=torch.bool, device=DEV)
    for e in (1, 2):
        assert out[0, sees, e].isnan().all() and lse[0, sees, e].isnan().all()
        assert (out[0, ~sees, e] == 0).all() and (lse[0, ~sees, e] == -np.inf).all()
    assert out[0, :, [0, 3]].isfinite().all() and lse[0, sees][:, [0, 3]].isfinite().all()


@pytest.mark.parametrize("length", [-1, -321, -2 ** 31])
@pytest.mark.parametrize("v_mode", [0, 1])
def test_any_negative_length_is_taken_as_none(length, v_mode):
    T, hkv, gq = 5, 1, 4
    case = build_decode_case([64 + 256 + 64 * 3, 700], hkv, gq, v_mode, seed=73)
    cache, _, hp, bp = case
    q, kd, vd = (to_dev_bf16(x) for x in draft(73, 2, T, hkv, gq))
    words = torch.from_numpy(mask_words(random_mask(np.random.default_rng(2), 2, T, "chain"))).to(DEV)
    ws = torch.empty(cache.tree_workspace_bytes(2, T, hp.shape[1]), dtype=torch.uint8, device=DEV)
    outs = []
    for n in (0, length):
        ws.fill_(0xFF)                                     # what is not written reads as NaN
        outs.append(cache.tree_attention(0, q, kd, vd, words, dev([n, 700]), hp, bp, synth.sm_scale(), workspace=ws))
        assert cache.get_status() == (0 if n == 0 else osc.STATUS_BAD_SEQLEN)
    assert torch.equal(outs[0], outs[1]) and outs[0].isfinite().all()


@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("meta", ["f16", "u8"])
@pytest.mark.parametrize("sm", [1e-12, 1e-20, 1e-38, 1e-44])
def test_the_smallest_scales_give_the_mean(T, meta, sm):
    # every logit is 0 to float32, so each row is the mean of what it sees: rows of zeros, tiny, ordinary and large q
    lens, hkv, gq = [64 + 256 + 64 * 3 + 9], 1, 4
    case = build_decode_case(lens, hkv, gq, 0, seed=75, meta=meta)
    cache, _, hp, bp = case
    q, kd, vd = draft(75, 1, T, hkv, gq)
    q[0, :, 0] = 0
    q[0, :, 1] *= 2.0 ** -100
    mask = random_mask(np.random.default_rng(6), 1, T, "tree")
    lse = torch.zeros(1, T, gq, device=DEV)
    out = cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV), dev(lens), hp,
                               bp, sm, out_dtype=osc.OUT_FP32, lse=lse)
    assert cache.get_status() == 0
    compare(out, lse, case, lens, q, kd, vd, mask, [T], 0, sm)
