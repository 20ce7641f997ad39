"""Commit of accepted draft tokens: the pool's bytes are those of single appends."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    from gpu_cases import DEV, head_params, to_dev_bf16, tokens, upload_params, with_codebooks
import synth
from tree_cases import mask_words, random_mask


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=DEV)


def two_caches(lens, hkv, v_mode, meta, extra_tokens, seed=80, gq=4):
    """Twice the same prefilled cache, with room for extra_tokens more per request."""
    B = len(lens)
    width = max(1, max(-(-max(0, L + extra_tokens - 320) // 64) for L in lens))
    prm = head_params(seed, 0, hkv)
    if meta == osc.META_CB:
        prm = with_codebooks(seed, 0, prm)
    out = []
    hp = np.random.default_rng(1).permutation(B * width).astype(np.int32).reshape(B, width)
    bp = np.arange(5 * B, dtype=np.int32).reshape(B, 5)[:, ::-1].copy()
    for _ in range(2):
        c = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=gq * hkv, num_int2_pages=B * width,
                                           num_bf16_pages=5 * B, max_batch=B, max_splits=16, v_mode=v_mode,
                                           meta_format=meta), device=DEV)
        upload_params(c, 0, prm)
        kv = [tokens(seed, 0, hkv, max(L, 1), extra=r) for r, L in enumerate(lens)]
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        cat = [np.concatenate([x[i][:L] for x, L in zip(kv, lens)]) for i in range(2)]
        if cu[-1]:
            c.quantize_prefill(0, to_dev_bf16(cat[0]), to_dev_bf16(cat[1]), cu, hp, bp)
        out.append(c)
    return out, dev(hp), dev(bp)


def append_one_by_one(cache, kd, vd, lens, n, path, hp, bp):
    for r in range(len(lens)):
        for j in range(int(n[r])):
            i = int(path[r][j])
            cache.append_kv(0, kd[r, i][None].contiguous(), vd[r, i][None].contiguous(), dev([lens[r] + j]), hp[r:r + 1],
                            bp[r:r + 1])


def node_rows(seed, B, T, hkv):
    kv = [tokens(seed, 0, hkv, T, extra=40 + b) for b in range(B)]
    return to_dev_bf16(np.stack([x[0] for x in kv])), to_dev_bf16(np.stack([x[1] for x in kv]))


@pytest.mark.parametrize("meta", [0, 1, 2])
@pytest.mark.parametrize("v_mode", [0, 1])
def test_equals_single_appends(meta, v_mode):
    lens = [0, 1, 60, 64, 310, 319, 320, 321, 640, 1000]
    B, T, hkv = len(lens), 40, 2
    (a, b), hp, bp = two_caches(lens, hkv, v_mode, meta, T)
    kd, vd = node_rows(81, B, T, hkv)
    rng = np.random.default_rng(meta)
    n = rng.integers(0, 34, B)
    n[[0, 6]] = [33, 33]
    n[4] = 0
    path = np.stack([np.sort(rng.permutation(T)[:33]) for _ in range(B)])
    path[7, 1] = path[7, 0]                                # the same node twice
    a.commit_draft(0, kd, vd, dev(lens), dev(n), hp, bp, path=dev(path))
    append_one_by_one(b, kd, vd, lens, n, path, hp, bp)
    assert a.get_status() == b.get_status() == 0
    assert torch.equal(a.pool, b.pool)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 255, 256])
def test_without_a_path_up_to_the_whole_window(n):
    lens, hkv = [900, 200, 320], 1
    (a, b), hp, bp = two_caches(lens, hkv, 0, 0, 256)
    kd, vd = node_rows(82, 3, n, hkv)
    a.commit_draft(0, kd, vd, dev(lens), dev([n, n, max(0, n - 1)]), hp, bp)
    append_one_by_one(b, kd, vd, lens, [n, n, max(0, n - 1)], [np.arange(n)] * 3, hp, bp)
    assert a.get_status() == b.get_status() == 0
    assert torch.equal(a.pool, b.pool)


def test_bad_requests_nodes_and_pages_are_left_out():
    lens, hkv, T = [700, 700, 700, 700, 700], 1, 8
    (a, b), hp, bp = two_caches(lens, hkv, 0, 0, 64)
    kd, vd = node_rows(83, 5, T, hkv)
    path = np.tile(np.arange(6), (5, 1))
    before = a.pool.clone()
    for ln, n in (([-1] * 5, [3] * 5), (lens, [-1] * 5), (lens, [7] * 5), ([2 ** 31 - 2] * 5, [3] * 5)):
        a.commit_draft(0, kd, vd, dev(ln), dev(n), hp, bp, path=dev(path))
        assert a.get_status() == osc.STATUS_BAD_SEQLEN
        assert torch.equal(a.pool, before)
    path[1, 2], path[2, 0] = T, -1                         # these tokens stay out, the others go in
    hbad, bbad = hp.clone(), bp.clone()
    hbad[3, :] = hp.numel()
    bbad[4, :] = -1
    a.commit_draft(0, kd, vd, dev(lens), dev([6] * 5), hbad, bbad, path=dev(path))
    assert a.get_status() == osc.STATUS_BAD_TREE | osc.STATUS_BAD_PAGE
    for r in range(3):
        for j in range(6):
            if 0 <= path[r, j] < T:
                i = int(path[r, j])
                b.append_kv(0, kd[r, i][None].contiguous(), vd[r, i][None].contiguous(), dev([700 + j]), hp[r:r + 1],
                            bp[r:r + 1])
    assert torch.equal(a.pool, b.pool)
    a.commit_draft(0, kd, vd, dev([700 + 64 * 40] * 5), dev([1] * 5), hp, bp, path=dev(path))   # beyond the page table
    assert a.get_status() & osc.STATUS_BAD_SEQLEN
    assert torch.equal(a.pool, b.pool)
    vd[0, 1, 0, 5] = float("nan")
    a.commit_draft(0, kd, vd, dev([706, 0, 0, 0, 0]), dev([2, 0, 0, 0, 0]), hp, bp, path=dev(path))
    assert a.get_status() == osc.STATUS_NONFINITE
    for bad in (dict(layer=1), dict(path=dev(path)[:4]), dict(n_accept=dev([1] * 4)), dict(max_accept=9, path=None),
                dict(k_draft=kd.float()), dict(k_draft=kd.flatten()), dict(hist_pt=hp.cpu()), dict(v_draft=vd[:, :4]), dict(max_accept=0, path=None)):
        with pytest.raises(osc.OscarError):
            a.commit_draft(**{**dict(layer=0, k_draft=kd, v_draft=vd, seq_lens_before=dev(lens), n_accept=dev([1] * 5),
                                     hist_pt=hp, bf16_pt=bp, path=dev(path)), **bad})


def test_verify_steps_from_an_empty_cache():
    """The operators one after another, as a speculative decoder runs them: tables, layout, rope, attention of the
    drafted chain, commit. Each chain node's output is checked against a decode of the same tokens in the 64-bit
    reference, and the cache against single appends of the rotated rows."""
    from tree_cases import attend
    from gpu_cases import pool_from_device
    B, T, hkv, gq, steps = 3, 9, 2, 4, 6
    (c, ref), _, _ = two_caches([0] * B, hkv, 0, 0, 1, gq=gq)
    width = 8
    cfg = osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hkv * gq, num_int2_pages=B * width,
                          num_bf16_pages=5 * B, max_batch=B, max_splits=16)
    prm = head_params(80, 0, hkv)
    c, ref = osc.OscarCache(cfg, device=DEV), osc.OscarCache(cfg, device=DEV)
    upload_params(c, 0, prm)
    upload_params(ref, 0, prm)
    rng = np.random.default_rng(7)
    hist = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    bf = torch.full((B, 5), -1, dtype=torch.int32, device=DEV)
    fi, fb = dev(rng.permutation(B * width)), dev(rng.permutation(5 * B))
    rings = dev([3, B * width, 2, 5 * B])
    plan = osc.RopePlan(128, base=1e6)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    # prompts: their tables, then the bulk write
    prompt = dev([300, 321, 700])
    _, cu, slots = c.build_tables(lens, prompt, hist, bf, fi, fb, rings, max_tokens=2000)
    k, v = tokens(84, 0, hkv, int(cu[-1]))
    k, v = to_dev_bf16(k), to_dev_bf16(v)
    osc.rope(plan, k, None, slots[:int(cu[-1]), 0].contiguous(), q_out=k)
    c.quantize_prefill(0, k, v, cu, hist, bf)
    ref.quantize_prefill(0, k, v, cu, hist, bf)
    lens = prompt
    for step in range(steps):
        q = to_dev_bf16(rng.standard_normal((B, T, hkv * gq, 128)) * 0.3)
        kd, vd = node_rows(100 + step, B, T, hkv)
        parents = np.stack([np.maximum(np.arange(T) - 1 - (rng.random(T) < 0.3), -1) for _ in range(B)]).astype(np.int32)
        mask, pos = c.tree_layout(parents, lens)
        osc.rope(plan, q.view(B * T, hkv * gq, 128), kd.view(B * T, hkv, 128), pos.view(-1), q_out=q.view(B * T, hkv * gq, 128),
                 k_out=kd.view(B * T, hkv, 128))
        out = c.tree_attention(0, q, kd, vd, mask, lens, hist, bf, synth.sm_scale(), out_dtype=osc.OUT_FP32)
        pm = pool_from_device(c, 0)
        seen = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=-1, bitorder="little")[..., :T].astype(bool)
        for b in range(B):
            x = [t[b].double().cpu().numpy() for t in (q, kd, vd)]
            o, _, bound, _ = attend(pm, prm, int(lens[b]), hist[b].cpu().numpy(), bf[b].cpu().numpy(), True, *x, seen[b],
                                    synth.sm_scale())
            assert (np.abs(out[b].double().cpu().numpy() - o) <= bound + 2.0 ** -24 * np.abs(o)).all()
        # accept the path to a random node
        n, path = np.zeros(B, np.int32), np.zeros((B, T), np.int32)
        for b in range(B):
            i = int(rng.integers(0, T))
            way = np.flatnonzero(seen[b, i])
            n[b], path[b, :len(way)] = len(way), way
        new = lens + dev(n)
        c.build_tables(lens, new, hist, bf, fi, fb, rings)
        c.commit_draft(0, kd, vd, lens, dev(n), hist, bf, path=dev(path))
        append_one_by_one(ref, kd, vd, lens.tolist(), n, path, hist, bf)
        lens = new
        assert c.get_status() == ref.get_status() == 0
        assert torch.equal(c.pool, ref.pool)
    # finished: every page is free again
    c.build_tables(lens, [0] * B, hist, bf, fi, fb, rings)
    assert rings[1] == B * width and rings[3] == 5 * B and (hist == -1).all() and (bf == -1).all()
    assert sorted(fi.tolist()) == list(range(B * width)) and sorted(fb.tolist()) == list(range(5 * B))
    assert c.get_status() == 0


def test_verify_step_on_another_stream_and_in_a_graph():
    # the calls of a step with stream=, and captured and replayed, leave the same bits as in a row on the current stream
    B, T, hkv, gq = 2, 6, 2, 4
    cfg = osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hkv * gq, num_int2_pages=B * 8, num_bf16_pages=5 * B,
                          max_batch=B, max_splits=16)
    prm = head_params(81, 0, hkv)
    rng = np.random.default_rng(9)
    q = to_dev_bf16(rng.standard_normal((B, T, hkv * gq, 128)) * 0.3)
    kd, vd = node_rows(90, B, T, hkv)
    k, v = (to_dev_bf16(x) for x in tokens(85, 0, hkv, 900))
    parents, path, n = dev([[-1, 0, 0, 1, 3, 2]] * B), dev([[0, 1, 3, 4, 0, 0]] * B), dev([4, 2])
    plan = osc.RopePlan(128)
    start, prompt = dev([0, 0]), dev([340, 560])

    def fresh():
        c = osc.OscarCache(cfg, device=DEV)
        upload_params(c, 0, prm)
        s = dict(c=c, hist=torch.full((B, 8), -1, dtype=torch.int32, device=DEV), bf=torch.full((B, 5), -1, dtype=torch.int32, device=DEV),
                 fi=dev(np.arange(B * 8)), fb=dev(np.arange(5 * B)), rings=dev([0, B * 8, 0, 5 * B]), lens=prompt.clone())
        _, cu, _ = c.build_tables(start, prompt, s["hist"], s["bf"], s["fi"], s["fb"], s["rings"])
        c.quantize_prefill(0, k, v, cu, s["hist"], s["bf"])
        s["new"] = s["lens"] + n
        return s

    def step(s, stream=None):
        c = s["c"]
        c.build_tables(s["lens"], s["new"], s["hist"], s["bf"], s["fi"], s["fb"], s["rings"], stream=stream)
        mask, pos = c.tree_layout(parents, s["lens"], stream=stream)
        qr, kr = osc.rope(plan, q.view(B * T, -1, 128), kd.view(B * T, -1, 128), pos.view(-1), stream=stream)
        s["out"] = c.tree_attention(0, qr.view(q.shape), kr.view(kd.shape), vd, mask, s["lens"], s["hist"], s["bf"], synth.sm_scale(),
                                    stream=stream)
        c.commit_draft(0, kr.view(kd.shape), vd, s["lens"], n, s["hist"], s["bf"], path=path, stream=stream)

    plain, other, graphed = fresh(), fresh(), fresh()
    step(plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(other, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graphed)
    assert not torch.equal(graphed["c"].pool, plain["c"].pool)   # captured, not run (no page is taken: the rings stay)
    g.replay()
    torch.cuda.synchronize()
    for s in (other, graphed):
        assert s["c"].get_status() == 0
        for key in ("hist", "bf", "fi", "fb", "rings", "out"):
            assert torch.equal(s[key], plain[key]), key
        assert torch.equal(s["c"].pool, plain["c"].pool)
