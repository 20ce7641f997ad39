"""Attention of drafted trees over the mixed cache against the oracle in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    from gpu_cases import DEV, build_decode_case, pool_from_device, queries, to_dev_bf16, tokens
import synth
from tree_cases import attend, attend_rounded, mask_words, random_mask


def draft(seed, B, T, hkv, gq, scale=1.0):
    """q [B, T, Hq, d], k, v [B, T, Hkv, d] float32 of bf16 values."""
    q = np.stack([queries(seed, 0, hkv, gq, batch=T, extra=50 + 7919 * b) for b in range(B)])
    kv = [tokens(seed, 0, hkv, T, extra=90 + b) for b in range(B)]
    return synth.bf16_round(q * scale), np.stack([x[0] for x in kv]), np.stack([x[1] for x in kv])


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=DEV)


def compare(out, lse, case, lens, q, kd, vd, mask, n, v_mode, sm):
    cache, prm, hp, bp = case
    pm = pool_from_device(cache, 0)
    got, lg = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
    eps = torch.finfo(out.dtype).eps / 2
    for b in range(len(lens)):
        k = int(n[b])
        o, l, bound, lb = attend(pm, prm, int(lens[b]), hp[b], bp[b], v_mode == 0, *(x[b, :k].astype(np.float64)
                                 for x in (q, kd, vd)), mask[b, :k, :k], sm)
        off = np.abs(got[b, :k] - o)
        tol = bound + eps * np.abs(o) * (1 + 2 ** -6)
        assert (off <= tol).all(), (b, (off / tol).max())
        if lg is not None:
            fin = np.isfinite(l)
            assert np.array_equal(np.isfinite(lg[b, :k]), fin) and (lg[b, :k][~fin] == -np.inf).all()
            assert (np.abs(lg[b, :k][fin] - l[fin]) <= lb[fin]).all()


@pytest.mark.parametrize("meta", ["f16", "u8", "cb"])
@pytest.mark.parametrize("v_mode", [0, 1])
@pytest.mark.parametrize("gq,T", [(4, 5), (1, 64), (8, 17), (2, 130)])
def test_formats_heads_and_trees(meta, v_mode, gq, T):
    lens, hkv = [64 + 256 + 64 * 9 + 21, 700], 2
    case = build_decode_case(lens, hkv, gq, v_mode, seed=60, meta=meta)
    rng = np.random.default_rng(T)
    q, kd, vd = draft(60, 2, T, hkv, gq)
    mask = random_mask(rng, 2, T, "tree")
    n = np.array([T, max(1, T - 3)])
    cache, _, hp, bp = case
    for dt in (osc.OUT_FP32, osc.OUT_BF16):
        out = torch.full((2, T, hkv * gq, 128), -77.0, dtype=torch.float32 if dt else torch.bfloat16, device=DEV)
        lse = torch.full((2, T, hkv * gq), -77.0, device=DEV)
        cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                             dev(lens), hp, bp, synth.sm_scale(), n_draft=dev(n), out=out, out_dtype=dt, lse=lse)
        assert cache.get_status() == 0
        compare(out, lse, case, lens, q, kd, vd, mask, n, v_mode, synth.sm_scale())
        assert (out[1, n[1]:] == -77).all() and (lse[1, n[1]:] == -77).all()   # rows behind the last node stay


@pytest.mark.parametrize("lens", [[0, 1, 63], [64, 65, 128], [319, 320, 321], [383, 384, 385], [448, 449, 577], [2000, 40, 5000]])
@pytest.mark.parametrize("kind", ["tree", "random", "none"])
@pytest.mark.parametrize("T", [9, 40])                     # rows of one tile and of two
def test_lengths_and_empty_rows(lens, kind, T):
    hkv, gq = 1, 4
    case = build_decode_case([max(x, 1) for x in lens], hkv, gq, 0, seed=61)
    rng = np.random.default_rng(5)
    q, kd, vd = draft(61, 3, T, hkv, gq)
    mask = random_mask(rng, 3, T, kind)
    cache, _, hp, bp = case
    lse = torch.zeros(3, T, 4, device=DEV)
    out = cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                               dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32, lse=lse)
    assert cache.get_status() == 0
    compare(out, lse, case, lens, q, kd, vd, mask, [T] * 3, 0, synth.sm_scale())
    if lens[0] == 0:                                       # a row that sees nothing
        empty = torch.from_numpy(~mask[0].any(-1)).to(DEV)
        assert (out[0][empty] == 0).all() and (lse[0][empty] == -np.inf).all()


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 255, 256])
def test_numbers_of_nodes(T):
    lens, hkv, gq = [777], 1, 4
    case = build_decode_case(lens, hkv, gq, 0, seed=62)
    q, kd, vd = draft(62, 1, T, hkv, gq)
    mask = random_mask(np.random.default_rng(T), 1, T, "chain")
    cache, _, hp, bp = case
    out = cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                               dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    assert cache.get_status() == 0
    compare(out, None, case, lens, q, kd, vd, mask, [T], 0, synth.sm_scale())


@pytest.mark.parametrize("scale", [8.0, 1 / 8.0])
@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("T", [24, 33])
def test_peaked_and_diffuse_logits(scale, aligned, T):
    lens, hkv, gq = [64 + 256 + 64 * 40 + 5], 2, 4
    case = build_decode_case(lens, hkv, gq, 0, seed=63)
    q, kd, vd = draft(63, 1, T, hkv, gq)
    if aligned:                                            # queries along keys of several pages: late, growing maxima
        k, _ = tokens(63, 0, hkv, lens[0], extra=1)
        for i in range(T):
            for h in range(hkv):
                q[0, i, h * gq + 1] = synth.bf16_round(0.05 * (1 + i) * k[64 + 79 * i, h])
    mask = random_mask(np.random.default_rng(1), 1, T, "tree")
    cache, _, hp, bp = case
    sm = synth.sm_scale() * scale
    out = cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                               dev(lens), hp, bp, sm, out_dtype=osc.OUT_FP32)
    assert cache.get_status() == 0
    compare(out, None, case, lens, q, kd, vd, mask, [T], 0, sm)


@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("up", [-60, 1, 60, 100])
def test_power_of_two_query_scales_change_nothing(T, up):
    # q 2^up against sm_scale 2^-up: the same logits. The kernel's own scale of the rotated rows is a power of two too,
    # so every rounding falls alike and the results are the same bits.
    lens, hkv, gq = [64 + 256 + 64 * 5 + 9], 1, 4
    cache, _, hp, bp = build_decode_case(lens, hkv, gq, 0, seed=65)
    q, kd, vd = (to_dev_bf16(x) for x in draft(65, 1, T, hkv, gq))
    mask = torch.from_numpy(mask_words(random_mask(np.random.default_rng(3), 1, T, "tree"))).to(DEV)
    args = (kd, vd, mask, dev(lens), hp, bp)
    plain = cache.tree_attention(0, q, *args, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    scaled = cache.tree_attention(0, (q.float() * 2.0 ** up).bfloat16(), *args, synth.sm_scale() * 2.0 ** -up,
                                  out_dtype=osc.OUT_FP32)
    assert cache.get_status() == 0 and torch.equal(plain, scaled)


def test_three_tiles_and_short_drafts():
    # 65 nodes x 4 heads are three row tiles; drafts that end in the first, at its end, in the second and the third
    lens, hkv, gq, T = [700, 800, 900, 1000, 640], 1, 4, 65
    case = build_decode_case(lens, hkv, gq, 0, seed=66)
    rng = np.random.default_rng(6)
    q, kd, vd = draft(66, 5, T, hkv, gq)
    mask = random_mask(rng, 5, T, "tree")
    n = np.array([5, 32, 33, 65, 0])
    cache, _, hp, bp = case
    out = torch.full((5, T, 4, 128), -77.0, device=DEV)
    lse = torch.full((5, T, 4), -77.0, device=DEV)
    cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                         dev(lens), hp, bp, synth.sm_scale(), n_draft=dev(n), out=out, out_dtype=osc.OUT_FP32, lse=lse)
    assert cache.get_status() == 0
    compare(out, lse, case, lens, q, kd, vd, mask, n, 0, synth.sm_scale())
    for b in range(5):
        assert (out[b, n[b]:] == -77).all() and (lse[b, n[b]:] == -77).all()


def test_long_context_and_error_size():
    # 20K tokens over many splits: the outputs are small means of large values, and the error is what the stated
    # roundings make, nothing more
    lens, hkv, gq, T = [20011], 1, 4, 24
    case = build_decode_case(lens, hkv, gq, 0, seed=64)
    q, kd, vd = draft(64, 1, T, hkv, gq)
    mask = random_mask(np.random.default_rng(2), 1, T, "tree")
    cache, prm, hp, bp = case
    args = [to_dev_bf16(x) for x in (q, kd, vd)] + [torch.from_numpy(mask_words(mask)).to(DEV), dev(lens), dev(hp), dev(bp)]
    ref, sd = attend_rounded(pool_from_device(cache, 0), prm, lens[0], hp[0], bp[0], *(x[0].astype(np.float64) for x in (q, kd, vd)),
                             mask[0], synth.sm_scale())

    def check(out):
        compare(out, None, case, lens, q, kd, vd, mask, [T], 0, synth.sm_scale())
        off = np.abs(out[0].double().cpu().numpy() - ref)
        # a rotated query channel within float32's error of an fp16 tie may round the other way: 2^-10 of one of 128
        # products of the logits, a tenth of a deviation of the weights' rounding
        assert (off <= 8.2 * sd + 2.0 ** -18 * np.abs(ref) + 2.0 ** -21).all(), (off / sd).max()

    out = cache.tree_attention(0, *args, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    check(out)
    again = cache.tree_attention(0, *args, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    assert torch.equal(out, again)                         # no order of summation is left to chance
    need = 1 * T * gq * 2 * 528                            # two slots per row: the history in one piece
    ws = torch.empty(-(-need // 256) * 256, dtype=torch.uint8, device=DEV)
    small = cache.tree_attention(0, *args, synth.sm_scale(), out_dtype=osc.OUT_FP32, workspace=ws)
    check(small)
    with pytest.raises(osc.OscarError) as e:
        cache.tree_attention(0, *args, synth.sm_scale(), workspace=ws[:need - 1])
    assert e.value.code == osc.ERR_INVALID_ARG
    assert cache.get_status() == 0


@pytest.mark.parametrize("T", [20, 40])
def test_compact_metadata_rounds_neither_keys_nor_values(T):
    lens, hkv, gq = [6011], 1, 4
    case = build_decode_case(lens, hkv, gq, 0, seed=67, meta="u8")
    q, kd, vd = draft(67, 1, T, hkv, gq)
    mask = random_mask(np.random.default_rng(4), 1, T, "tree")
    cache, prm, hp, bp = case
    out = cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                               dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    assert cache.get_status() == 0
    ref, sd = attend_rounded(pool_from_device(cache, 0), prm, lens[0], hp[0], bp[0], *(x[0].astype(np.float64) for x in (q, kd, vd)),
                             mask[0], synth.sm_scale(), compact=True)
    off = np.abs(out[0].double().cpu().numpy() - ref)      # the bound of the test above
    assert (off <= 8.2 * sd + 2.0 ** -18 * np.abs(ref) + 2.0 ** -21).all(), (off / sd).max()


def test_many_rows_in_explicit_mode():
    # enough rows for the merge's 32-row CTAs, of requests with history and without, and a draft that ends inside one
    lens, hkv, gq, T, B = [700, 90] * 5, 2, 8, 251, 10
    case = build_decode_case(lens, hkv, gq, 1, seed=68)
    q, kd, vd = draft(68, B, T, hkv, gq)
    mask = random_mask(np.random.default_rng(7), B, T, "tree")
    n = np.array([T, T, 77, 0] + [T] * 6)
    cache, prm, hp, bp = case
    out = torch.full((B, T, hkv * gq, 128), -77.0, device=DEV)
    lse = torch.full((B, T, hkv * gq), -77.0, device=DEV)
    cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV),
                         dev(lens), hp, bp, synth.sm_scale(), n_draft=dev(n), out=out, out_dtype=osc.OUT_FP32, lse=lse)
    assert cache.get_status() == 0
    for b in range(B):
        assert (out[b, n[b]:] == -77).all() and (lse[b, n[b]:] == -77).all()
    few = [1, 2]
    part = lambda x: np.asarray(x.cpu() if isinstance(x, torch.Tensor) else x)[few]   # noqa: E731
    compare(out[few], lse[few], (cache, prm, part(hp), part(bp)), [lens[b] for b in few], q[few], kd[few], vd[few], mask[few],
            n[few], 1, synth.sm_scale())
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[4:]).all()


def test_one_node_is_one_decode_step():
    # a single node over the cache and itself, before it is appended: with the recent window not yet full nothing is
    # demoted, so the tokens are those of oscar_decode_step
    lens, hkv, gq = [200, 290], 2, 4
    case = build_decode_case(lens, hkv, gq, 0, seed=65)
    cache, _, hp, bp = case
    q, kd, vd = (to_dev_bf16(x) for x in draft(65, 2, 1, hkv, gq))
    mask = torch.ones(2, 1, 1, dtype=torch.int64, device=DEV)
    out = cache.tree_attention(0, q, kd, vd, mask, dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    ref = cache.decode_step(0, q[:, 0].contiguous(), kd[:, 0].contiguous(), vd[:, 0].contiguous(), dev(lens), dev(hp),
                            dev(bp), synth.sm_scale(), out_dtype=osc.OUT_FP32)
    # both keep the BF16 rows' weights to about 2^-16 and everything else in float32
    assert (out[:, 0] - ref).abs().max() <= 2.0 ** -13 * ref.abs().max()


def test_nonfinite_drafts_reach_only_the_rows_that_see_them():
    lens, hkv, gq, T = [900, 500], 1, 4, 70
    case = build_decode_case(lens, hkv, gq, 0, seed=66)
    cache, _, hp, bp = case
    q, kd, vd = draft(66, 2, T, hkv, gq)
    mask = random_mask(np.random.default_rng(3), 2, T, "tree")
    words = torch.from_numpy(mask_words(mask)).to(DEV)
    qd, k2, v2 = (to_dev_bf16(x) for x in (q, kd, vd))
    for b, j, what, val in ((0, 3, k2, np.nan), (0, 20, v2, np.inf), (0, 65, v2, np.nan), (1, 69, k2, -np.inf), (1, 0, v2, -np.inf)):
        what[b, j, 0, 17] = val
    out = cache.tree_attention(0, qd, k2, v2, words, dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32,
                               n_draft=dev([T, 69]))
    assert cache.get_status() == osc.STATUS_NONFINITE
    hurt = np.zeros((2, T), bool)
    for b, j in ((0, 3), (0, 20), (0, 65), (1, 0)):        # (1, 69) is behind the last node
        hurt[b] |= mask[b, :, j]
    got = out.cpu().numpy()
    assert np.isfinite(got[0][~hurt[0]]).all() and np.isfinite(got[1, :69][~hurt[1, :69]]).all()
    for b, j in ((0, 20), (0, 65), (1, 0)):                # the value's channel is NaN or infinite
        assert not np.isfinite(got[b, :69][mask[b, :69, j]][..., 17]).any()
    # the unhurt rows are what they are without the bad nodes
    clean = cache.tree_attention(0, qd, to_dev_bf16(kd), to_dev_bf16(vd), words, dev(lens), hp, bp, synth.sm_scale(),
                                 out_dtype=osc.OUT_FP32, n_draft=dev([T, 69])).cpu().numpy()
    for b, k in ((0, T), (1, 69)):
        assert np.array_equal(got[b, :k][~hurt[b, :k]], clean[b, :k][~hurt[b, :k]])
    assert cache.get_status() == 0


def test_stale_rows_behind_the_length_do_not_count():
    # ring and history rows that hold NaN, behind the tokens of a short request
    lens, hkv, gq, T = [330], 1, 4, 6
    case = build_decode_case(lens, hkv, gq, 0, seed=67)
    cache, _, hp, bp = case
    bf = cache.bf16_pages(0).view(torch.bfloat16).reshape(-1, hkv, 2, 64, 128)
    blk = cache.int2_pages(0)
    blk[int(hp[0, 0]), :, 4096 + 8 * 10:4608] = 0xff       # scale and zero of rows 10.. as NaN
    blk[int(hp[0, 0]), :, 4608 + 8 * 10:5120] = 0xff
    q, kd, vd = draft(67, 1, T, hkv, gq)
    mask = random_mask(np.random.default_rng(4), 1, T, "chain")
    args = [to_dev_bf16(x) for x in (q, kd, vd)] + [torch.from_numpy(mask_words(mask)).to(DEV)]
    out = cache.tree_attention(0, *args, dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    compare(out, None, case, lens, q, kd, vd, mask, [T], 0, synth.sm_scale())
    short = [100]                                          # 36 tokens in the ring; the rest of it is stale
    bf[bp[0, 1].item(), :, :, 36:] = float("nan")
    bf[bp[0, 2].item()] = float("inf")
    out = cache.tree_attention(0, *args, dev(short), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    compare(out, None, case, short, q, kd, vd, mask, [T], 0, synth.sm_scale())
    assert cache.get_status() == 0


def test_bad_pages_and_lengths_are_reported_and_skipped():
    lens, hkv, gq, T = [64 + 256 + 64 * 6, 600], 1, 4, 9
    case = build_decode_case(lens, hkv, gq, 0, seed=68)
    cache, prm, hp, bp = case
    q, kd, vd = draft(68, 2, T, hkv, gq)
    mask = random_mask(np.random.default_rng(4), 2, T, "chain")
    args = [to_dev_bf16(x) for x in (q, kd, vd)] + [torch.from_numpy(mask_words(mask)).to(DEV)]
    run = lambda ln, h, b, **kw: cache.tree_attention(0, *args, dev(ln), h, b, synth.sm_scale(), out_dtype=osc.OUT_FP32, **kw)  # noqa: E731
    want = run(lens, hp, bp)
    for value in (-1, cache.cfg.num_int2_pages, 2 ** 30):
        bad = hp.copy()
        bad[0, 3] = value
        got = run(lens, bad, bp)
        assert cache.get_status() == osc.STATUS_BAD_PAGE
        assert torch.equal(got[1], want[1]) and torch.isfinite(got).all()
    bad = bp.copy()
    bad[1, 2] = cache.cfg.num_bf16_pages
    got = run(lens, hp, bad)
    assert cache.get_status() == osc.STATUS_BAD_PAGE
    assert torch.equal(got[0], want[0]) and torch.isfinite(got).all()
    got = run([lens[0], -3], hp, bp)                       # a negative length is taken as 0
    assert cache.get_status() == osc.STATUS_BAD_SEQLEN
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], run([lens[0], 0], hp, bp)[1])
    got = run([lens[0] + 64 * 50, lens[1]], hp, bp)        # longer than its page table: its pages count
    assert cache.get_status() == osc.STATUS_BAD_SEQLEN
    assert torch.equal(got[1], want[1]) and torch.isfinite(got).all()
    got = run(lens, hp, bp, n_draft=dev([T + 1, T]))
    assert cache.get_status() == osc.STATUS_BAD_TREE
    assert torch.equal(got, want)


def test_argument_checks():
    case = build_decode_case([400], 1, 4, 0, seed=69)
    cache, _, hp, bp = case
    q, kd, vd = (to_dev_bf16(x) for x in draft(69, 1, 3, 1, 4))
    ok = dict(layer=0, q=q, k_draft=kd, v_draft=vd, mask=torch.zeros(1, 3, 1, dtype=torch.int64, device=DEV),
              seq_lens=dev([400]), hist_pt=hp, bf16_pt=bp, sm_scale=0.1)
    cache.tree_attention(**ok)
    for bad in (dict(layer=1), dict(layer=-1), dict(q=q.float()), dict(q=q[:, :2]), dict(q=q.flatten()), dict(q=q.cpu()),
                dict(seq_lens=dev([400]).cpu()), dict(lse=torch.zeros(1, 3, 4, 1, device=DEV)), dict(k_draft=kd[:, :2]),
                dict(v_draft=vd.transpose(0, 1)), dict(mask=ok["mask"][:, :2]), dict(mask=ok["mask"].int()),
                dict(seq_lens=dev([1, 2])), dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(sm_scale=float("inf")),
                dict(out_dtype=2), dict(n_draft=dev([1, 2])), dict(out=torch.zeros(1, 3, 4, 128, device=DEV)),
                dict(workspace=torch.empty(4096, dtype=torch.uint8, device=DEV)[:256])):
        with pytest.raises(osc.OscarError):
            cache.tree_attention(**{**ok, **bad})
    big = torch.zeros(1, 257, 4, 128, dtype=torch.bfloat16, device=DEV)
    kb = torch.zeros(1, 257, 1, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(osc.OscarError) as e:
        cache.tree_attention(0, big, kb, kb, torch.zeros(1, 257, 5, dtype=torch.int64, device=DEV), dev([400]), hp, bp, 0.1)
    assert e.value.code == osc.ERR_UNSUPPORTED
    for bad in ((2, 3, 1), (1, 0, 1), (1, 3, -1), (1, 257, 1)):
        with pytest.raises(osc.OscarError):
            cache.tree_workspace_bytes(*bad)


def test_streams_and_two_captured_graphs():
    lens, hkv, gq, T = [1500, 900], 2, 4, 12
    case = build_decode_case(lens, hkv, gq, 0, seed=70)
    cache, _, hp, bp = case
    q, kd, vd = (to_dev_bf16(x) for x in draft(70, 2, T, hkv, gq))
    words = torch.from_numpy(mask_words(random_mask(np.random.default_rng(4), 2, T, "tree"))).to(DEV)
    ln, hp, bp = dev(lens), dev(hp), dev(bp)
    want = cache.tree_attention(0, q, kd, vd, words, ln, hp, bp, synth.sm_scale())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    cache.tree_attention(0, q, kd, vd, words, ln, hp, bp, synth.sm_scale(), out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graphs, outs = [], []
    for half in range(2):                                  # a request each, a workspace each
        ws = torch.empty(cache.tree_workspace_bytes(1, T, hp.shape[1]), dtype=torch.uint8, device=DEV)
        o = torch.zeros_like(want[:1])
        part = [x[half:half + 1] for x in (q, kd, vd, words, ln, hp, bp)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.tree_attention(0, *part, synth.sm_scale(), out=o, workspace=ws)
        graphs.append((g, ws, part))
        outs.append(o)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _, _), st in zip(graphs, side):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    alone = [cache.tree_attention(0, *part, synth.sm_scale()) for _, _, part in graphs]
    for o, a in zip(outs, alone):
        assert torch.equal(o, a)
    assert cache.get_status() == 0


def test_captured_after_a_join_and_after_a_copy():
    # the call's launch is a programmatic dependent of what is before it on the stream: here two kernels, a copy, a memset
    lens, hkv, gq, T = [500], 1, 4, 40
    cache, _, hp, bp = build_decode_case(lens, hkv, gq, 0, seed=69)
    q, kd, vd = (to_dev_bf16(x) for x in draft(69, 1, T, hkv, gq))
    words = torch.from_numpy(mask_words(random_mask(np.random.default_rng(8), 1, T, "tree"))).to(DEV)
    ln, hp, bp = dev(lens), dev(hp), dev(bp)
    plain = cache.tree_attention(0, q, kd, vd, words, ln, hp, bp, synth.sm_scale())
    src, zero = q.clone(), torch.zeros_like(q)
    side, outs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        q.mul_(0.0)
        with torch.cuda.stream(side):
            zero.zero_()
        main.wait_stream(side)
        outs.append(cache.tree_attention(0, zero, kd, vd, words, ln, hp, bp, synth.sm_scale()))
        q.copy_(src)
        outs.append(cache.tree_attention(0, q, kd, vd, words, ln, hp, bp, synth.sm_scale()))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert cache.get_status() == 0 and torch.equal(outs[1], plain)
    assert torch.equal(outs[0], cache.tree_attention(0, zero, kd, vd, words, ln, hp, bp, synth.sm_scale()))
