"""The row operators, the prompt attention, the cache and the decode step together, as a layer of a served model calls them:
prompts' raw projections are normed and rotated, attended and placed in the cache, and further tokens are decoded from it. While
a request has 320 tokens or fewer its cache holds BF16 rows alone, so every step has a 64-bit value to be held against.

Bounds. Rows against the 64-bit norm and rotation: layer_cases.py. Attention over the rows as they were rounded: prompt_cases.py;
the decode step takes its weights as two bf16 parts and merges up to five partials, each a few steps of 2^-24: less than the
2^-8 that the bound gives to a weight's rounding.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import layer_cases as L  # noqa: E402
import prompt_cases as C  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    import gpu_cases as G
    DEV = torch.device("cuda:0")

SM, EPS = 1.0 / 128 ** 0.5, 1e-5


class Layer:
    """One layer's weights, cache and page tables for prompts of `lens` tokens."""

    def __init__(self, lens, hkv, gq, axes, layout, seed):
        self.B, self.hkv, self.hq, self.layout, self.axes = len(lens), hkv, hkv * gq, layout, axes
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g, self.w = g, (1 + 0.3 * torch.randn(2, 128, generator=g, device=DEV)).bfloat16()
        self.plan = osc.RopePlan(64, base=1e6, scale=1.1, axes=None if axes == 1 else np.arange(32) % axes)
        self.cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=self.hq, num_int2_pages=1,
                                                    num_bf16_pages=5 * self.B, max_batch=self.B), device=DEV)
        G.upload_params(self.cache, 0, G.head_params(seed, 0, hkv))
        self.bf = torch.randperm(5 * self.B, generator=torch.Generator().manual_seed(seed)).int().view(self.B, 5).to(DEV)
        self.hist = torch.full((self.B, 1), -1, dtype=torch.int32, device=DEV)

    def raw(self, n):
        x = torch.randn(n, self.hq + 2 * self.hkv, 128, generator=self.g, device=DEV).bfloat16()
        return x.split((self.hq, self.hkv, self.hkv), 1)                 # views of one projection

    def positions(self, at):
        """Positions of tokens at places `at` of their sequences: the place itself, or one number an axis."""
        return at if self.axes == 1 else torch.stack([at // (i + 1) for i in range(self.axes)]).int()

    def prompt(self, q, k, v, cu, at):
        qn, kn = osc.norm_rope(self.plan, q, k, self.positions(at), self.w[0], self.w[1], eps=EPS, layout=self.layout)
        out = self.cache.prompt_attention(qn, kn, v, cu, SM)
        self.cache.quantize_prefill(0, kn, v.contiguous(), cu, self.hist, self.bf, total_tokens=len(q))
        return qn, kn, out

    def step(self, q, k, v, lens, q_out):
        return self.cache.decode_step_rope(0, self.plan, q, k, v, lens, self.hist, self.bf, SM, self.w[0], self.w[1], eps=EPS,
                                           positions=None if self.axes == 1 else self.positions(lens), layout=self.layout,
                                           q_out=q_out)

    def rows(self, r, n):
        """The cache's first n keys and values of request r."""
        pages = self.cache.bf16_pages(0).view(torch.bfloat16).view(5 * self.B, self.hkv, 2, 64, 128)
        kv = torch.cat([pages[p] for p in self.bf[r].tolist()], 2)[:, :, :n]
        return kv[:, 0].transpose(0, 1), kv[:, 1].transpose(0, 1)


CASES = [([1, 130, 300], 2, 4, 1, 0), ([64, 63, 0, 315], 1, 8, 3, 1), ([7] * 40, 8, 1, 1, 1)]   # lens, hkv, gq, axes, layout


@pytest.mark.parametrize("lens,hkv,gq,axes,layout", CASES)
def test_prompt_then_steps(lens, hkv, gq, axes, layout):
    m = Layer(lens, hkv, gq, axes, layout, 3)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    at = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(DEV)
    q, k, v = m.raw(len(at))
    qn, kn, out = m.prompt(q, k, v, cu, at)
    for got, x, w in ((qn, q, m.w[0]), (kn, k, m.w[1])):
        L.near(got, *L.norm_rope(x, w, EPS, m.plan, m.positions(at).cpu(), layout))
    C.check(out, None, qn, kn, v, lens, cu[:-1].tolist(), SM)
    for r, n in enumerate(lens):
        ck, cv = m.rows(r, n)
        assert torch.equal(ck, kn[cu[r]:cu[r + 1]]) and torch.equal(cv, v[cu[r]:cu[r + 1]])
    now = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for _ in range(4):
        q, k, v = m.raw(m.B)
        q_out = torch.zeros(m.B, m.hq, 128, dtype=torch.bfloat16, device=DEV)
        out = m.step(q, k, v, now, q_out)
        pos = m.positions(now).cpu()
        now = now + 1
        got_k = torch.stack([m.rows(r, n)[0][-1] for r, n in enumerate(now.tolist())])
        for got, x, w in ((q_out, q, m.w[0]), (got_k, k, m.w[1])):
            L.near(got, *L.norm_rope(x, w, EPS, m.plan, pos, layout))
        for r, n in enumerate(now.tolist()):
            ck, cv = m.rows(r, n)
            assert torch.equal(cv[-1], v[r])
            full_q, full_out = torch.zeros(n, m.hq, 128, dtype=torch.bfloat16, device=DEV), torch.zeros_like(out[:1]).repeat(n, 1, 1)
            full_q[-1], full_out[-1] = q_out[r], out[r]
            C.check(full_out, None, full_q, ck, cv, [n], [0], SM, rows={n - 1})
    assert m.cache.get_status() == 0


def test_prompt_then_steps_in_a_graph():
    lens = [100, 5, 200]
    m = Layer(lens, 2, 4, 1, 0, 5)
    cu = torch.tensor([0, 100, 105, 305], dtype=torch.int32, device=DEV)
    at = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(DEV)
    first = [x.clone() for x in m.raw(305)]
    new = [[x.contiguous() for x in m.raw(3)] for _ in range(3)]
    q_out = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    start = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run():
        outs = [m.prompt(*first, cu, at)[2]]
        now = start.clone()
        for x in new:
            outs.append(m.step(*x, now, q_out))
            now = now + 1
        return outs

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for seed in range(3):                                                # new inputs in the same graph
        for x in (*first, *(y for step in new for y in step)):
            x.copy_(torch.randn(x.shape, generator=m.g, device=DEV))
        m.cache.pool.zero_()
        graph.replay()
        got, pool = [x.clone() for x in held], m.cache.pool.clone()
        m.cache.pool.zero_()
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(pool, m.cache.pool)
    assert m.cache.get_status() == 0


def test_gradient_of_the_rows_that_are_attended():
    # the gradient of sum(g . norm_rope(x)) and the forward pass agree along a random direction of x and w, in 64 bits: both are
    # within their bounds of the formulas, and the formulas' difference quotient is central and of third order
    m = Layer([50], 2, 4, 3, 1, 6)
    at = m.positions(torch.arange(50, dtype=torch.int32, device=DEV))
    q, k, _ = m.raw(50)
    gq, gk = torch.randn(q.shape, generator=m.g, device=DEV).bfloat16(), torch.randn(k.shape, generator=m.g, device=DEV).bfloat16()
    dq, dk, dwq, dwk = osc.norm_rope_backward(m.plan, q, k, at, gq, gk, m.w[0], m.w[1], eps=EPS, layout=1)
    for x, g, w, dx, dw in ((q, gq, m.w[0], dq, dwq), (k, gk, m.w[1], dk, dwk)):
        x64, w64, g64 = x.double().cpu(), w.double().cpu(), g.double().cpu()
        gen = torch.Generator().manual_seed(1)
        tx, tw, h = torch.randn(x64.shape, generator=gen).double(), torch.randn(128, generator=gen).double(), 1e-4

        def f(s):
            return (L.turned(L.normed(x64 + s * tx, w64 + s * tw, EPS)[0], m.plan, at.cpu(), 1)[0] * g64).sum()

        want = (f(h) - f(-h)) / (2 * h)
        # bounds of dx and dw, each entry times its direction's, and the quotient's third order: |f'''| h^2 / 6 with every
        # derivative of r below 16 r^3 |t|: far below 1e-6 of the sizes summed
        (rx, bx), (rw, bw) = L.norm_rope_grad(x, g, w, EPS, m.plan, at.cpu(), 1, 64)
        L.near(dx, rx, bx)
        size = (rx.abs() * tx.abs()).sum() + (rw.abs() * tw.abs()).sum()
        off = (bx * tx.abs()).sum() + (bw * tw.abs()).sum() + 1e-6 * size
        assert abs((dx.double().cpu() * tx).sum() + (dw.double().cpu() * tw).sum() - want) <= off


def far(n, heads, g):
    """Rows [n, heads, 128] of normal values, the last ones more than 2^32 bytes (and 2^31 elements) behind the first."""
    step = (2 ** 31 // (n - 1) + 16) // 8 * 8
    x = torch.empty((n - 1) * step + heads * 128, dtype=torch.bfloat16, device=DEV).as_strided((n, heads, 128), (step, 128, 1))
    return x.copy_(torch.randn(n, heads, 128, generator=g, device=DEV))


def test_rows_far_apart():
    g = torch.Generator(device=DEV).manual_seed(8)
    q, k, v, gq, gk = far(65, 4, g), far(65, 2, g), far(65, 2, g), far(65, 4, g), far(65, 2, g)
    plan, pos = osc.RopePlan(128), torch.arange(65, dtype=torch.int32, device=DEV)
    w = (1 + 0.3 * torch.randn(2, 128, generator=g, device=DEV)).bfloat16()
    near = [x.contiguous() for x in (q, k, v, gq, gk)]
    # the same bits as from rows side by side, which have their own tests
    for a, b in zip(osc.norm_rope(plan, q, k, pos, w[0], w[1]), osc.norm_rope(plan, *near[:2], pos, w[0], w[1])):
        assert torch.equal(a, b)
    for a, b in zip(osc.norm_rope_backward(plan, q, k, pos, gq, gk, w[0], w[1]),
                    osc.norm_rope_backward(plan, *near[:2], pos, *near[3:], w[0], w[1])):
        assert torch.equal(a, b)
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=2, num_q_heads=4, num_int2_pages=1, num_bf16_pages=325,
                                           max_batch=65), device=DEV)
    cu = torch.tensor([0, 65], dtype=torch.int32, device=DEV)
    assert torch.equal(cache.prompt_attention(q, k, v, cu, SM), cache.prompt_attention(*near[:3], cu, SM))
    bf = torch.arange(325, dtype=torch.int32, device=DEV)
    hist = torch.full((65, 1), -1, dtype=torch.int32, device=DEV)
    outs = []
    for rows in ((q, k, v), near[:3]):
        cache.pool.zero_()
        out = cache.append_kv_rope(0, plan, *rows, pos, hist, bf, w[0], w[1])
        outs.append((out, cache.pool.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert cache.get_status() == 0


def test_results_past_32_bits():
    # 270,000 prompts of one token with 64 heads: results past 2^31 elements; a token that sees itself alone has its own value
    n = 270_000
    g = torch.Generator(device=DEV).manual_seed(9)
    q = torch.empty(n, 64, 128, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    k, v = (torch.empty(n, 8, 128, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2))
    cache = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=8, num_q_heads=64, num_int2_pages=1, num_bf16_pages=5), device=DEV)
    out = cache.prompt_attention(q, k, v, torch.arange(n + 1, dtype=torch.int32, device=DEV), SM)
    assert cache.get_status() == 0
    for h in range(8):
        assert torch.equal(out[:, 8 * h:8 * h + 8], v[:, h:h + 1].expand(n, 8, 128))
