"""The drafted-token calls over windows other than 64 sink and 256 recent tokens: no sink, several sink pages, long windows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    from gpu_cases import DEV, head_params, to_dev_bf16, tokens, upload_params
    from test_gpu_tree import dev, draft
import synth
from oracle import pool as P
from tree_cases import attend, mask_words, random_mask

WINDOWS = [(0, 64), (128, 192), (192, 1024)]


def built(lens, sink, recent, hkv, gq, v_mode=0, room=0, seed=90, copies=1):
    """Caches whose pools hold the oracle's bytes of the requests' tokens: (caches, params, hist_pt, bf16_pt, model)."""
    B, nbf = len(lens), (sink + recent) // 64
    width = max(1, max(-(-max(0, L + room - sink - recent) // 64) for L in lens))
    rng = np.random.default_rng(seed)
    hp = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    bp = rng.permutation(B * nbf).astype(np.int32).reshape(B, nbf)
    prm = head_params(seed, 0, hkv)
    pm = P.PoolModel(P.PoolGeometry(hkv=hkv, sink=sink, recent=recent), B * width, B * nbf)
    for r, L in enumerate(lens):
        if L:
            k, v = tokens(seed, 0, hkv, L, extra=r)
            P.prefill(pm, k, v, hp[r], bp[r], prm, v_mode == 0)
    caches = []
    for _ in range(copies):
        c = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hkv * gq, num_int2_pages=B * width,
                                           num_bf16_pages=B * nbf, max_batch=B, max_splits=16, sink=sink, recent=recent,
                                           v_mode=v_mode), device=DEV)
        upload_params(c, 0, prm)
        c.int2_pages(0).copy_(torch.from_numpy(pm.int2).reshape(c.int2_pages(0).shape))
        c.bf16_pages(0).copy_(torch.from_numpy(pm.bf16.view(np.uint8)).reshape(c.bf16_pages(0).shape))
        caches.append(c)
    return caches, prm, hp, bp, pm


def check(out, lse, pm, prm, lens, hp, bp, q, kd, vd, mask, v_mode, rows=slice(None)):
    for b, L in enumerate(lens):
        o, l, bound, lb = attend(pm, prm, int(L), hp[b], bp[b], v_mode == 0, *(x[b].astype(np.float64) for x in (q, kd, vd)),
                                 mask[b], synth.sm_scale())
        off = np.abs(out[b].double().cpu().numpy() - o)
        tol = bound + 2.0 ** -24 * np.abs(o) * (1 + 2 ** -6)
        assert (off <= tol)[rows].all(), (b, L, (off / tol)[rows].max())
        got, fin = lse[b].double().cpu().numpy(), np.isfinite(l)
        assert np.array_equal(np.isfinite(got), fin) and (np.abs(got - l)[fin & np.isfinite(got)] <= lb[fin]).all()


@pytest.mark.parametrize("sink,recent", WINDOWS)
@pytest.mark.parametrize("T", [9, 40])                     # rows of one tile and of two
@pytest.mark.parametrize("v_mode", [0, 1])
def test_tree_attention(sink, recent, T, v_mode):
    at = [0, 1, sink - 1, sink, sink + 1, sink + 63, sink + 65, sink + recent - 1, sink + recent, sink + recent + 1, sink + recent + 64,
          sink + recent + 65, sink + recent + 200]
    lens = sorted({x for x in at if x >= 0})
    hkv, gq = 1, 4
    (c,), prm, hp, bp, pm = built(lens, sink, recent, hkv, gq, v_mode)
    B = len(lens)
    q, kd, vd = draft(91, B, T, hkv, gq)
    mask = random_mask(np.random.default_rng(T), B, T, "tree")
    lse = torch.zeros(B, T, hkv * gq, device=DEV)
    args = [to_dev_bf16(x) for x in (q, kd, vd)] + [torch.from_numpy(mask_words(mask)).to(DEV), dev(lens), hp, bp, synth.sm_scale()]
    out = c.tree_attention(0, *args, out_dtype=osc.OUT_FP32, lse=lse)
    assert c.get_status() == 0
    check(out, lse, pm, prm, lens, hp, bp, q, kd, vd, mask, v_mode)


@pytest.mark.parametrize("T,gq", [(130, 1), (130, 4)])
def test_a_long_window_in_one_slot(T, gq):
    # the least workspace: 61 BF16 pages and the draft's three in one slot, NaN and infinity among the last ones' values
    sink, recent, hkv = 64, 64 * 60, 1
    lens = [sink + recent + 64 * 3 + 7, sink + 64 * 58 + 33]
    (c,), prm, hp, bp, pm = built(lens, sink, recent, hkv, gq)
    q, kd, vd = draft(92, 2, T, hkv, gq)
    mask = random_mask(np.random.default_rng(3), 2, T, "tree")
    words = torch.from_numpy(mask_words(mask)).to(DEV)
    rows = T * gq
    rows = -(-rows // 8) * 8 if rows <= 128 else -(-rows // 128) * 128
    ws = torch.empty(-(-2 * rows * 2 * 528 // 256) * 256, dtype=torch.uint8, device=DEV)
    qd, k2, v2 = (to_dev_bf16(x) for x in (q, kd, vd))
    clean, lse = [], torch.zeros(2, T, hkv * gq, device=DEV)
    for w in (ws, None):
        clean.append(c.tree_attention(0, qd, k2, v2, words, dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32, lse=lse,
                                      workspace=w))
        assert c.get_status() == 0
        few = slice(0, T, 13)
        check(clean[-1], lse, pm, prm, lens, hp, bp, q, kd, vd, mask, 0, few)
    for b, j, val in ((0, 3, np.nan), (0, 66, np.inf), (1, 129, -np.inf)):
        v2[b, j, 0, 31] = val
    hurt = torch.from_numpy(np.stack([mask[0, :, 3] | mask[0, :, 66], mask[1, :, 129]])).to(DEV)
    for w, want in zip((ws, None), clean):
        out = c.tree_attention(0, qd, k2, v2, words, dev(lens), hp, bp, synth.sm_scale(), out_dtype=osc.OUT_FP32, workspace=w)
        assert c.get_status() == osc.STATUS_NONFINITE
        assert torch.equal(out[~hurt], want[~hurt]) and not out[hurt][..., 31].isfinite().any()
    # a row of the last page but one, behind the length of the second request: stale, and not looked at
    page = int(bp[1, 60])
    c.bf16_pages(0).view(torch.bfloat16).reshape(-1, hkv, 2, 64, 128)[page] = float("nan")
    out = c.tree_attention(0, qd, *(to_dev_bf16(x) for x in (kd, vd)), words, dev(lens), hp, bp, synth.sm_scale(),
                           out_dtype=osc.OUT_FP32, workspace=ws)
    assert c.get_status() == 0 and torch.equal(out[1], clean[0][1])


def test_the_longest_window_and_one_page_more():
    for pages, ok in ((2040, True), (2041, False)):
        c = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=1, num_bf16_pages=1,
                                           max_batch=1, max_splits=1, sink=64, recent=64 * (pages - 1)), device=DEV)
        q = torch.randn(1, 2, 1, 128, device=DEV).bfloat16()
        bp = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
        args = (0, q, q, q, torch.ones(1, 2, 1, dtype=torch.int64, device=DEV), dev([50]), dev([[0]]), bp, 0.1)
        if ok:
            assert c.tree_attention(*args).isfinite().all() and c.get_status() == 0
        else:
            with pytest.raises(osc.OscarError) as e:
                c.tree_attention(*args)
            assert e.value.code == osc.ERR_UNSUPPORTED


@pytest.mark.parametrize("sink,recent", WINDOWS)
@pytest.mark.parametrize("v_mode", [0, 1])
def test_commit_equals_single_appends(sink, recent, v_mode):
    full = sink + recent
    at = [0, 1, sink - 1, sink, sink + 1, full - 40, full - 1, full, full + 1, full + 63, full + 130]
    lens = sorted({x for x in at if x >= 0})
    B, T, hkv = len(lens), 40, 2
    (a, b), _, hp, bp, _ = built(lens, sink, recent, hkv, 4, v_mode, room=64, copies=2)
    kv = [tokens(93, 0, hkv, T, extra=r) for r in range(B)]
    kd, vd = (to_dev_bf16(np.stack([x[i] for x in kv])) for i in range(2))
    rng = np.random.default_rng(sink)
    A = min(33, recent)
    n = rng.integers(0, A + 1, B)
    n[:2], n[-1] = A, A
    path = np.stack([np.sort(rng.permutation(T)[:A]) for _ in range(B)])
    hd, bd = dev(hp), dev(bp)
    a.commit_draft(0, kd, vd, dev(lens), dev(n), hd, bd, path=dev(path))
    for r in range(B):
        for j in range(int(n[r])):
            i = int(path[r, j])
            b.append_kv(0, kd[r, i][None].contiguous(), vd[r, i][None].contiguous(), dev([lens[r] + j]), hd[r:r + 1], bd[r:r + 1])
    assert a.get_status() == b.get_status() == 0
    assert torch.equal(a.pool, b.pool)


@pytest.mark.parametrize("recent", [64, 1024])
def test_commit_of_a_whole_window(recent):
    sink, T = 0, min(recent, 256)
    lens = [recent - 1, recent + 70, 3]
    (a, b), _, hp, bp, _ = built(lens, sink, recent, 1, 4, room=256, copies=2)
    kv = [tokens(94, 0, 1, T, extra=r) for r in range(3)]
    kd, vd = (to_dev_bf16(np.stack([x[i] for x in kv])) for i in range(2))
    hd, bd = dev(hp), dev(bp)
    path = dev(np.tile(np.arange(recent) % T, (3, 1)))     # more tokens than nodes where the window is long
    n = [recent if r < 2 else 5 for r in range(3)]
    if recent > 256:
        n = [256, 256, 5]
        path = path[:, :256].contiguous()
    a.commit_draft(0, kd, vd, dev(lens), dev(n), hd, bd, path=path)
    for r in range(3):
        for j in range(n[r]):
            i = int(path[r, j])
            b.append_kv(0, kd[r, i][None].contiguous(), vd[r, i][None].contiguous(), dev([lens[r] + j]), hd[r:r + 1], bd[r:r + 1])
    assert a.get_status() == b.get_status() == 0
    assert torch.equal(a.pool, b.pool)


@pytest.mark.parametrize("sink,recent", WINDOWS + [(64, 256)])
@pytest.mark.parametrize("B", [1, 37, 4096])
def test_tables(sink, recent, B):
    nbf = (sink + recent) // 64
    up = lambda n: -(-n // 64)                             # noqa: E731
    counts = [lambda L: up(max(0, L - sink - recent)), lambda L: up(min(L, sink)) + up(min(max(L - sink, 0), recent))]
    width = 6
    rng = np.random.default_rng(B)
    caps = [width * B + 1, nbf * B + 2]
    tables = [np.full((B, width), -1, np.int32), np.full((B, nbf), -1, np.int32)]
    free = [rng.permutation(n).astype(np.int32) for n in caps]
    rings = [int(rng.integers(caps[0])), caps[0], int(rng.integers(caps[1])), caps[1]]
    c = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=caps[0], num_bf16_pages=caps[1],
                                       max_batch=1, max_splits=1, sink=sink, recent=recent), device=DEV)
    on = [dev(x) for x in (*tables, *free, rings)]
    lens = np.zeros(B, np.int64)
    edges = [x for x in (1, sink, sink + 1, sink + 64, sink + recent - 1, sink + recent, sink + recent + 1, sink + recent + 65,
                         sink + recent + 250) if x > 0]
    for step in range(5):
        new = rng.choice(edges, B) if step == 0 else np.minimum(lens + rng.choice([0, 1, 5, 64, 70], B), sink + recent + width * 64)
        if step > 1:
            new[rng.random(B) < 0.3] = 0
        slots, cu = [], [0]
        for e in range(2):
            head, count = rings[2 * e:2 * e + 2]
            took, back = 0, []
            for r in range(B):
                held, want = counts[e](int(lens[r])), counts[e](int(new[r]))
                if new[r] >= lens[r]:
                    for j in range(held, want):
                        tables[e][r, j] = free[e][(head + took) % caps[e]]
                        took += 1
                else:
                    back += tables[e][r, :held].tolist()
                    tables[e][r, :held] = -1
            for i, x in enumerate(back):
                free[e][(head + count + i) % caps[e]] = x
            rings[2 * e:2 * e + 2] = [(head + took) % caps[e], count - took + len(back)]
        for r in range(B):
            for pos in range(int(lens[r]), int(new[r])):
                seg = P.segment_of(pos, int(new[r]), c_geo(sink, recent))
                if seg == "history":
                    slots.append((pos, 1, tables[0][r, (pos - sink) // 64], (pos - sink) % 64))
                else:
                    page, row = P.bf16_location(pos, seg, tables[1][r], c_geo(sink, recent))
                    slots.append((pos, 0 if seg == "sink" else 2, page, row))
            cu.append(len(slots))
        out = torch.full((len(slots) + 2, 4), -7, dtype=torch.int32, device=DEV)
        _, got_cu, _ = c.build_tables(dev(lens), dev(new), *on, slots=out)
        lens = new.astype(np.int64)
        assert c.get_status() == 0
        for x, y in zip(on, (*tables, *free, np.array(rings))):
            assert np.array_equal(x.cpu().numpy(), y)
        assert np.array_equal(got_cu.cpu().numpy(), cu) and (out[len(slots):] == -7).all()
        assert np.array_equal(out[:len(slots)].cpu().numpy(), np.array(slots, np.int32).reshape(-1, 4))
        if B > 1000 and step == 2:
            break


def c_geo(sink, recent):
    return P.PoolGeometry(hkv=1, sink=sink, recent=recent)
