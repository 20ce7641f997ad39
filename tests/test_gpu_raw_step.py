"""Appends and decode steps from raw projections: the new key and the queries against the 64-bit norm and rotation
(bounds: layer_cases.py), everything else bit by bit against the calls that take them ready-made."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import layer_cases as L  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    import gpu_cases as G
    DEV = torch.device("cuda:0")

SM = 1.0 / 128 ** 0.5


def raw(g, B, hq, hkv, strided=True):
    """q, k, v as views of one projection's rows, with a little room behind each row."""
    x = torch.randn(B, (hq + 2 * hkv) * 128 + 16, generator=g, device=DEV).bfloat16()
    x[:, 3::128] *= 16
    q, k, v = x[:, : hq * 128], x[:, hq * 128:(hq + hkv) * 128], x[:, (hq + hkv) * 128:(hq + 2 * hkv) * 128]
    out = [t.unflatten(1, (-1, 128)) for t in (q, k, v)]
    return out if strided else [t.contiguous() for t in out]


def new_rows(cache, lens, bf16_pt):
    """The K and V rows [B, Hkv, 128] that hold the tokens at positions lens."""
    pages = cache.bf16_pages(0).view(torch.bfloat16).view(cache.cfg.num_bf16_pages, cache.cfg.num_kv_heads, 2, 64, 128)
    slot = [n if n < 64 else 64 + (n - 64) % 256 for n in lens]
    at = [int(bf16_pt[r, s // 64]) for r, s in enumerate(slot)]
    rows = torch.stack([pages[p, :, :, s % 64] for p, s in zip(at, slot)])
    return rows[:, :, 0], rows[:, :, 1]


def pair(lens, hkv, gq, v_mode, seed, **kw):
    """Two caches with the same contents and room for one more token."""
    a, _, hist, bf = G.build_decode_case([n + 1 for n in lens], hkv, gq, v_mode, seed, **kw)
    b = osc.OscarCache(a.cfg, device=DEV, pool=a.pool.clone())
    b.set_decode_algo(kw.get("algo", 0))
    return a, b, hist, bf


CASES = [  # lens, hkv, gq, v_mode, meta, algo, rot, layout, axes
    ([0, 5, 63, 64, 319], 2, 4, 0, "f16", 1, 128, 0, 1),
    ([320, 321, 700], 2, 4, 1, "f16", 1, 64, 1, 3),
    ([1500], 8, 4, 0, "f16", 1, 128, 0, 1),
    ([383, 384], 1, 8, 0, "u8", 1, 24, 0, 3),
    ([640, 10, 2000], 4, 1, 1, "cb", 1, 20, 0, 1),
    ([900, 333], 2, 2, 0, "f16", 0, 2, 1, 1),
    ([20 * i for i in range(42)], 8, 1, 1, "f16", 1, 64, 0, 1),      # many CTAs: the fragments come from L2
    ([900, 333], 2, 2, 0, "f16", 2, 128, 1, 3),
]


@pytest.mark.parametrize("lens,hkv,gq,v_mode,meta,algo,rot,layout,axes", CASES)
@pytest.mark.parametrize("normed", [True, False])
def test_against_ready_made_rows(lens, hkv, gq, v_mode, meta, algo, rot, layout, axes, normed):
    B, hq = len(lens), hkv * gq
    a, b, hist, bf = pair(lens, hkv, gq, v_mode, 70 + gq, meta=meta, algo=algo)
    g = torch.Generator(device=DEV).manual_seed(B)
    q, k, v = raw(g, B, hq, hkv)
    qw, kw = (1 + 0.3 * torch.randn(2, 128, generator=g, device=DEV)).bfloat16()
    plan = osc.RopePlan(rot, base=1e6, scale=1.125, axes=None if axes == 1 else np.arange(rot // 2) % axes)
    pos = None if axes == 1 else torch.randint(0, 10 ** 6, (axes, B), generator=g, device=DEV, dtype=torch.int32)
    norm = dict(q_weight=qw, k_weight=kw, eps=1e-5) if normed else dict(eps=None)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    before = a.pool.clone()

    q_out = a.append_kv_rope(0, plan, q, k, v, sl, hist, bf, positions=pos, layout=layout, **norm)
    assert a.get_status() == 0
    krow, vrow = new_rows(a, lens, bf)
    host_pos = np.array(lens) if pos is None else pos.cpu()
    for got, x, w in ((q_out, q, qw), (krow, k, kw)):
        if normed:
            L.near(got, *L.norm_rope(x, w, 1e-5, plan, host_pos, layout))
        else:
            want, size = L.turned(x.double().cpu(), plan, host_pos, layout)
            L.near(got, want, L.rounded(want, size * 2.0 ** -20.5, torch.bfloat16))
    assert torch.equal(vrow, v)
    # the same bytes as an append of those rows, also without queries
    b.append_kv(0, krow.contiguous(), v.contiguous(), sl, hist, bf)
    assert torch.equal(a.pool, b.pool)
    a.pool.copy_(before)
    assert a.append_kv_rope(0, plan, None, k, v, sl, hist, bf, positions=pos, layout=layout, **norm) is None
    assert torch.equal(a.pool, b.pool)
    # and the same results as a decode step with those rows
    a.pool.copy_(before)
    b.pool.copy_(before)
    lse, lse_b = torch.zeros(B, hq, device=DEV), torch.zeros(B, hq, device=DEV)
    mine = torch.zeros_like(q_out)
    out = a.decode_step_rope(0, plan, q, k, v, sl, hist, bf, SM, positions=pos, layout=layout, q_out=mine,
                             out_dtype=osc.OUT_FP32, lse=lse, **norm)
    want = b.decode_step(0, q_out, krow.contiguous(), v.contiguous(), sl, hist, bf, SM, out_dtype=osc.OUT_FP32, lse=lse_b)
    assert a.get_status() == 0 and b.get_status() == 0
    assert torch.equal(mine, q_out) and torch.equal(out, want) and torch.equal(lse, lse_b) and torch.equal(a.pool, b.pool)


def test_weights_off_16_bytes():
    a, b, hist, bf = pair([500], 2, 4, 0, 85, algo=1)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = raw(g, 1, 8, 2)
    w = (1 + 0.3 * torch.randn(2, 129, generator=g, device=DEV)).bfloat16()
    plan, sl = osc.RopePlan(128), np.array([500], np.int32)
    x = a.decode_step_rope(0, plan, q, k, v, sl, hist, bf, SM, w[0, 1:], w[1, 1:])
    y = b.decode_step_rope(0, plan, q, k, v, sl, hist, bf, SM, w[0, 1:].clone(), w[1, 1:].clone())
    assert torch.equal(x, y) and torch.equal(a.pool, b.pool)


def test_shared_prefix():
    lens, hkv, gq = [1100, 1200], 2, 4
    a, b, hist, bf = pair(lens, hkv, gq, 0, 81, shared_prefix=576, algo=1)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = raw(g, 2, 8, hkv)
    plan, sl = osc.RopePlan(128), torch.tensor(lens, dtype=torch.int32, device=DEV)
    q_out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    out = a.decode_step_rope(0, plan, q, k, v, sl, hist, bf, SM, q_out=q_out, shared_hist_pages=8)
    krow, _ = new_rows(a, lens, bf)
    want = b.decode_step(0, q_out, krow.contiguous(), v.contiguous(), sl, hist, bf, SM, shared_hist_pages=8)
    assert torch.equal(out, want) and torch.equal(a.pool, b.pool)


def test_in_place_streams_and_graphs():
    lens, hkv, gq = [500, 40], 2, 4
    a, b, hist, bf = pair(lens, hkv, gq, 0, 82, algo=1)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = raw(g, 2, 8, hkv, strided=False)
    plan = osc.RopePlan(128)
    sl, hist, bf = (torch.as_tensor(x, dtype=torch.int32, device=DEV) for x in (lens, hist, bf))
    before, q0 = a.pool.clone(), q.clone()
    want_q = a.append_kv_rope(0, plan, q, k, v, sl, hist, bf)
    want_pool = a.pool.clone()
    a.pool.copy_(before)
    a.append_kv_rope(0, plan, q, k, v, sl, hist, bf, q_out=q)              # in place
    assert torch.equal(q, want_q) and torch.equal(a.pool, want_pool)
    q.copy_(q0)
    want = b.decode_step_rope(0, plan, q, k, v, sl, hist, bf, SM)
    out, q_out = torch.zeros_like(q), torch.zeros_like(q)
    s = torch.cuda.Stream()
    a.pool.copy_(before)
    s.wait_stream(torch.cuda.current_stream())
    a.decode_step_rope(0, plan, q, k, v, sl, hist, bf, SM, q_out=q_out, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(q_out, want_q) and torch.equal(a.pool, want_pool)
    graph = torch.cuda.CUDAGraph()
    pos = sl.clone()
    with torch.cuda.graph(graph):
        # projections, positions, tables and last the lengths from the kernels straight before
        q2, k2, pos2, hist2, bf2 = q * 1, k * 1, pos + 0, hist + 0, bf + 0
        a.decode_step_rope(0, plan, q2, k2, v, sl + 0, hist2, bf2, SM, positions=pos2, q_out=q_out, out=out)
    for _ in range(3):
        a.pool.copy_(before)
        out.zero_()
        q_out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(q_out, want_q) and torch.equal(a.pool, want_pool)


def test_status():
    a, _, hist, bf = pair([100, 30], 2, 4, 0, 83, algo=1)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = raw(g, 2, 8, 2)
    plan = osc.RopePlan(128, axes=np.zeros(64, int))
    sl = torch.tensor([100, 30], dtype=torch.int32, device=DEV)
    call = lambda **kw: a.append_kv_rope(0, plan, **{**dict(q=q, k=k, v=v, seq_lens_before=sl, hist_pt=hist, bf16_pt=bf),   # noqa: E731
                                                     **kw})
    zero = call(positions=torch.tensor([[0, 7]], dtype=torch.int32, device=DEV))
    assert a.get_status() == 0
    got = call(positions=torch.tensor([[-4, 7]], dtype=torch.int32, device=DEV))
    assert a.get_status() == osc.STATUS_BAD_SEQLEN and torch.equal(got, zero)
    for name, x in (("q", q), ("k", k), ("v", v)):
        bad = x.clone()
        bad[1, 1, 5] = float("nan")
        got = call(**{name: bad}, positions=torch.tensor([[0, 7]], dtype=torch.int32, device=DEV))
        assert a.get_status() == osc.STATUS_NONFINITE
        if name == "q":
            assert got[1, 1].isnan().all() and torch.equal(got[0], zero[0]) and torch.equal(got[1, 2:], zero[1, 2:])
        else:
            assert torch.equal(got, zero)
    before = a.pool.clone()
    call(seq_lens_before=torch.tensor([-1, 30], dtype=torch.int32, device=DEV))
    assert a.get_status() == osc.STATUS_BAD_SEQLEN
    krow, _ = new_rows(a, [100, 30], bf)
    call()
    assert a.get_status() == 0 and before.shape == a.pool.shape and torch.equal(new_rows(a, [100, 30], bf)[0][1], krow[1])


def test_refusals():
    a, _, hist, bf = pair([100, 30], 2, 4, 0, 84)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = raw(g, 2, 8, 2)
    w = torch.ones(128, device=DEV).bfloat16()
    good = dict(layer=0, plan=osc.RopePlan(128), q=q, k=k, v=v, seq_lens_before=np.array([100, 30], np.int32), hist_pt=hist,
                bf16_pt=bf)
    odd = torch.zeros(2, 8 * 128 + 4, dtype=torch.bfloat16, device=DEV)[:, 4:].unflatten(1, (8, 128))
    for bad in (dict(q=q[:, :7]), dict(k=q), dict(v=v.float()), dict(q=q.float()), dict(k=None), dict(v=None), dict(q=odd),
                dict(q=q.transpose(1, 2)), dict(layer=1), dict(layout=2), dict(eps=0.0), dict(q_weight=w.float()),
                dict(k_weight=w[:64]), dict(plan=osc.RopePlan(130)), dict(q_out=q), dict(bf16_pt=bf[:1]),
                dict(hist_pt=hist[:1]), dict(positions=np.zeros(3, np.int32)), dict(seq_lens_before=np.zeros(3, np.int32)),
                dict(plan=osc.RopePlan(64, axes=np.arange(32) % 2), positions=np.zeros(2, np.int32))):
        with pytest.raises(osc.OscarError):
            a.append_kv_rope(**{**good, **bad})
        with pytest.raises(osc.OscarError):
            a.decode_step_rope(**{**good, **bad}, sm_scale=SM)
    for bad in (dict(q=None), dict(sm_scale=0.0), dict(out=torch.zeros(2, 8, 128, device=DEV)), dict(shared_hist_pages=99)):
        with pytest.raises(osc.OscarError):
            a.decode_step_rope(**{**good, **dict(sm_scale=SM), **bad})
    empty = dict(q=q[:0], k=k[:0], v=v[:0], seq_lens_before=np.zeros(0, np.int32), hist_pt=hist[:0], bf16_pt=bf[:0])
    assert a.append_kv_rope(**{**good, **empty}).shape == (0, 8, 128)
    assert a.decode_step_rope(**{**good, **empty}, sm_scale=SM).shape == (0, 8, 128)


def test_lengths_from_the_kernel_just_before():
    # each step's lengths and tables come from kernels right in front of it, in a graph that is replayed
    lens, hkv, gq, steps = [300, 63, 318, 1000], 2, 4, 6
    a, b, hist, bf = pair([n + steps for n in lens], hkv, gq, 0, 87, algo=1)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = [raw(g, 4, 8, hkv) for _ in range(steps)]
    plan, start = osc.RopePlan(128), torch.tensor(lens, dtype=torch.int32, device=DEV)
    hist, bf = (torch.as_tensor(t, dtype=torch.int32, device=DEV) for t in (hist, bf))
    now, tables = start.clone(), torch.zeros_like(bf)
    before = a.pool.clone()

    def run():
        outs = []
        for q, k, v in x:
            torch.add(bf, 0, out=tables)
            outs.append(a.decode_step_rope(0, plan, q, k, v, now, hist, tables, SM, out_dtype=osc.OUT_FP32))
            torch.add(now, 1, out=now)
            tables.fill_(-1)
        return outs

    want = []
    for i, (q, k, v) in enumerate(x):
        torch.cuda.synchronize()
        want.append(b.decode_step_rope(0, plan, q, k, v, start + i, hist, bf, SM, out_dtype=osc.OUT_FP32))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(20):
        a.pool.copy_(before)
        now.copy_(start)
        graph.replay()
        assert all(torch.equal(p, r) for p, r in zip(outs, want)) and torch.equal(a.pool, b.pool)
    assert a.get_status() == 0 and b.get_status() == 0
