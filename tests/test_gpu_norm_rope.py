"""Rotary positions with several axes, the norm with the rotation in one pass, and its gradient, on the GPU against
64-bit formulas. References, bounds and their derivation: layer_cases.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import layer_cases as L  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

DIMS = [(128, 128), (128, 64), (64, 24), (64, 20), (256, 256), (96, 2), (80, 80), (512, 512), (512, 2), (512, 16), (34, 6), (2, 2)]


def plan_of(rot, axes, **kw):
    return osc.RopePlan(rot, base=1e6, axes=None if axes == 1 else np.arange(rot // 2) % axes, **kw)


def positions(g, axes, n, top=200_000):
    p = torch.randint(0, top, (axes, n), generator=g, device=DEV, dtype=torch.int32)
    p[:, :1] = 2 ** 31 - 1
    p[-1, -1:] = 0
    return p[0] if axes == 1 else p


def rows(g, n, heads, dim, dtype):
    x = torch.randn(n, heads, dim, generator=g, device=DEV)
    x[..., : max(1, dim // 16)] *= 8
    return x.to(L.DTYPES[dtype])


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dim,rot", DIMS)
@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_axes(dtype, dim, rot, layout):
    axes = min(3, rot // 2)
    g = torch.Generator(device=DEV).manual_seed(dim + rot)
    x, pos = rows(g, 37, 9, dim, dtype), positions(g, max(2, axes), 37)
    if axes == 1:
        pos = pos[:1]
    plan = osc.RopePlan(rot, base=1e6, axes=np.arange(rot // 2) % axes, scale=1.25)
    for inverse in (False, True):
        q, k = osc.rope(plan, x[:, :6], x[:, 6:], pos, layout=layout, inverse=inverse)
        for got, rows_in in ((q, x[:, :6]), (k, x[:, 6:])):
            want, size = L.turned(rows_in.double().cpu(), plan, pos.cpu(), layout, inverse)
            L.near(got, want, L.rounded(want, size * 2.0 ** -20.5, x.dtype))
            assert torch.equal(got[..., rot:], rows_in[..., rot:])


@pytest.mark.parametrize("layout", [0, 1])
def test_equal_axes_are_one_axis(layout):
    g = torch.Generator(device=DEV).manual_seed(2)
    x = rows(g, 301, 5, 128, "bf16")
    pos = torch.randint(0, 10 ** 6, (301,), generator=g, device=DEV, dtype=torch.int32)
    pos[7] = -1
    one, three = osc.RopePlan(96, base=1e6), osc.RopePlan(96, base=1e6, axes=np.repeat([0, 1, 2], 16))
    a, b = torch.zeros_like(x), torch.zeros_like(x)
    osc.rope(one, x, None, pos, layout=layout, q_out=a)
    osc.rope(three, x, None, pos.repeat(3, 1), layout=layout, q_out=b)
    assert torch.equal(a, b)
    w = rows(g, 1, 1, 128, "bf16")[0, 0]
    osc.norm_rope(one, x, None, pos, w, layout=layout, q_out=a)
    osc.norm_rope(three, x, None, pos.repeat(3, 1), w, layout=layout, q_out=b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dim,rot", DIMS)
@pytest.mark.parametrize("dtype", list(L.DTYPES))
def test_norm_and_gradient(dtype, dim, rot, layout):
    axes = min(3, rot // 2) if dim != 128 else 1
    g = torch.Generator(device=DEV).manual_seed(dim + rot + 1)
    N, hq, hkv = 37, 6, 3
    x, gr = rows(g, N, hq + hkv, dim, dtype), rows(g, N, hq + hkv, dim, dtype)
    q, k, gq, gk = x[:, :hq], x[:, hq:], gr[:, :hq].contiguous(), gr[:, hq:]
    qw, kw = (1 + 0.3 * rows(g, 1, 2, dim, "f32")[0]).to(x.dtype)
    pos, plan = positions(g, axes, N), plan_of(rot, axes, scale=1.25)
    qo, ko = osc.norm_rope(plan, q, k, pos, qw, kw, eps=1e-5, layout=layout)
    for got, xx, w in ((qo, q, qw), (ko, k, kw)):
        L.near(got, *L.norm_rope(xx, w, 1e-5, plan, pos.cpu(), layout), "forward")
    dq, dk, dqw, dkw = osc.norm_rope_backward(plan, q, k, pos, gq, gk, qw, kw, eps=1e-5, layout=layout)
    for dx, dw, xx, gg, w in ((dq, dqw, q, gq, qw), (dk, dkw, k, gk, kw)):
        (ex, bx), (ew, bw) = L.norm_rope_grad(xx, gg, w, 1e-5, plan, pos.cpu(), layout, N * hq)
        L.near(dx, ex, bx, "dx")
        L.near(dw, ew, bw, "dw")
    # in place: the rows' buffer, the gradient's
    y, gy = x.clone(), gr.clone()
    osc.norm_rope(plan, y[:, :hq], y[:, hq:], pos, qw, kw, eps=1e-5, layout=layout, q_out=y[:, :hq], k_out=y[:, hq:])
    assert torch.equal(y[:, :hq], qo) and torch.equal(y[:, hq:], ko)
    got = osc.norm_rope_backward(plan, q, k, pos, gy[:, :hq], gy[:, hq:], qw, kw, eps=1e-5, layout=layout, dq=gy[:, :hq],
                                 dk=gy[:, hq:])
    assert all(torch.equal(a, b) for a, b in zip(got, (dq, dk, dqw, dkw)))
    y = x.clone()
    osc.norm_rope_backward(plan, y[:, :hq], y[:, hq:], pos, gq, gk, qw, kw, eps=1e-5, layout=layout, dq=y[:, :hq], dk=y[:, hq:])
    assert torch.equal(y[:, :hq], dq) and torch.equal(y[:, hq:], dk)


@pytest.mark.parametrize("N", [1, 2, 5, 305, 3000, 20011])
def test_numbers_of_tokens(N):
    g = torch.Generator(device=DEV).manual_seed(N)
    q, gq = rows(g, N, 2, 64, "f32"), rows(g, N, 2, 64, "f32")
    k, gk = rows(g, N, 1, 64, "f32"), rows(g, N, 1, 64, "f32")
    pos, plan = positions(g, 1, N), osc.RopePlan(64)
    qo, ko = osc.norm_rope(plan, q, k, pos)
    L.near(qo, *L.norm_rope(q, None, 1e-6, plan, pos.cpu(), 0))
    L.near(ko, *L.norm_rope(k, None, 1e-6, plan, pos.cpu(), 0))
    dq, dk, dqw, dkw = osc.norm_rope_backward(plan, q, k, pos, gq, gk)
    for dx, dw, x, gg in ((dq, dqw, q, gq), (dk, dkw, k, gk)):
        # a lane's chain: its share of the CTAs' rows, 202 CTAs at least and 16 groups of rows in each
        (ex, bx), (ew, bw) = L.norm_rope_grad(x, gg, None, 1e-6, plan, pos.cpu(), 0, N * 2)
        L.near(dx, ex, bx)
        L.near(dw, ew, bw)
    again = osc.norm_rope_backward(plan, q, k, pos, gq, gk)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dqw, dkw)))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("shift,token", [(0, 9 * 128), (8, 1160), (4, 1156), (1, 1153), (3, 9 * 131)])
def test_strides_and_alignments(layout, shift, token):
    buf = torch.randn(20 * token + 16, device=DEV).bfloat16()
    head = 131 if token == 9 * 131 else 128
    x = buf.as_strided((20, 9, 128), (token, head, 1), shift)
    pos = torch.arange(20, dtype=torch.int32, device=DEV) * 977
    plan = osc.RopePlan(96)
    w = (1 + torch.rand(129, device=DEV)).bfloat16()[1:]                 # off 16 bytes too
    q, _ = osc.norm_rope(plan, x, None, pos, w, layout=layout)
    L.near(q, *L.norm_rope(x, w, 1e-6, plan, pos.cpu(), layout))
    t = torch.zeros(9, 20, 128, dtype=torch.bfloat16, device=DEV)        # heads outermost
    osc.norm_rope(plan, x, None, pos, w, layout=layout, q_out=t.transpose(0, 1))
    one = torch.tensor(2.0 ** -7)                                        # another width of access: other sums, one step at most
    assert ((t.transpose(0, 1).float() - q.float()).abs() <= one * q.float().abs() + 1e-30).all()
    dq, _, dw, _ = osc.norm_rope_backward(plan, x, None, pos, t.transpose(0, 1), None, w, layout=layout)
    (ex, bx), (ew, bw) = L.norm_rope_grad(x, t.transpose(0, 1), w, 1e-6, plan, pos.cpu(), layout, 180)
    L.near(dq, ex, bx)
    L.near(dw, ew, bw)


@pytest.mark.parametrize("axes", [1, 3])
def test_padded_rows_stay(axes):
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, gq, gk = (rows(g, 6, h, 128, "bf16") for h in (4, 2, 4, 2))
    pos = torch.tensor([5, -1, 7, -1, -3, 0], dtype=torch.int32, device=DEV)
    if axes == 3:
        pos = torch.stack([pos.clamp(min=0), pos, pos.clamp(min=1)])
    plan = plan_of(128, axes)
    q[1], gk[3] = float("nan"), float("inf")                             # padded rows may hold anything
    outs = [torch.full_like(t, -3.0) for t in (q, k)]
    osc.norm_rope(plan, q, k, pos, q_out=outs[0], k_out=outs[1])
    grads = [torch.full_like(t, -3.0) for t in (q, k)]
    _, _, dqw, dkw = osc.norm_rope_backward(plan, q, k, pos, gq, gk, dq=grads[0], dk=grads[1])
    live = torch.tensor([0, 2, 5])
    for out, grad, dw, x, gg in ((outs[0], grads[0], dqw, q, gq), (outs[1], grads[1], dkw, k, gk)):
        for i in (1, 3, 4):
            assert (out[i] == -3).all() and (grad[i] == -3).all()
        p = pos.cpu()[..., live]
        want, bound = L.norm_rope(x[live.to(DEV)], None, 1e-6, plan, p, 0)
        L.near(out[live.to(DEV)], want, bound)
        (ex, bx), (ew, bw) = L.norm_rope_grad(x[live.to(DEV)], gg[live.to(DEV)], None, 1e-6, plan, p, 0, 24)
        L.near(grad[live.to(DEV)], ex, bx)
        L.near(dw, ew, bw)


def test_rows_do_not_reach_each_other():
    g = torch.Generator(device=DEV).manual_seed(6)
    x, gr = rows(g, 5, 3, 128, "bf16"), rows(g, 5, 3, 128, "bf16")
    pos, plan = torch.arange(5, dtype=torch.int32, device=DEV), osc.RopePlan(128)
    want, dwant = osc.norm_rope(plan, x, None, pos)[0], osc.norm_rope_backward(plan, x, None, pos, gr, None)[0]
    bad = x.clone()
    bad[2, 1, 5], bad[3, 0] = float("nan"), 0.0                          # zeros: the norm of a zero row is zero
    got, dgot = osc.norm_rope(plan, bad, None, pos)[0], osc.norm_rope_backward(plan, bad, None, pos, gr, None)[0]
    assert got[2, 1].isnan().all() and (got[3, 0] == 0).all() and dgot[2, 1].isnan().all() and dgot[3, 0].isfinite().all()
    same = torch.ones(5, 3, dtype=torch.bool, device=DEV)
    same[2, 1] = same[3, 0] = False
    assert torch.equal(got[same], want[same]) and torch.equal(dgot[same], dwant[same])


@pytest.mark.parametrize("layout", [0, 1])
def test_gradient_against_differences(layout):
    # f = <c, y(x, w)>; along d, (f(x + e d) - f(x - e d)) / 2e = <dx, d> + O(e^2), with the 64-bit forward
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, c, d = (torch.randn(9, 5, 64, generator=gen, device=DEV) for _ in range(3))
    w, dwd = torch.rand(64, generator=gen, device=DEV) + 0.5, torch.randn(64, generator=gen, device=DEV)
    pos = torch.randint(0, 10 ** 5, (9,), generator=gen, device=DEV, dtype=torch.int32)
    plan = osc.RopePlan(32, scale=1.25)
    f = lambda a, b: (c.double().cpu() * L.turned(L.normed(a, b, 1e-6)[0], plan, pos.cpu(), layout)[0]).sum()   # noqa: E731
    dx, _, dw, _ = osc.norm_rope_backward(plan, x, None, pos, c, None, w, layout=layout)
    e = 1e-4
    x64, w64 = x.double().cpu(), w.double().cpu()
    by_x = (f(x64 + e * d.double().cpu(), w64) - f(x64 - e * d.double().cpu(), w64)) / (2 * e)
    by_w = (f(x64, w64 + e * dwd.double().cpu()) - f(x64, w64 - e * dwd.double().cpu())) / (2 * e)
    size = (dx.double().abs() * d.double().abs()).sum().item() + (dw.double().abs() * dwd.double().abs()).sum().item()
    # third derivatives of the normed rows are below 2^7 of the sums of |c| |d|, times e^2 / 6; float32's part as derived
    assert abs(by_x - (dx.double() * d.double()).sum().item()) <= size * (2.0 ** 7 * e * e / 6 + 2.0 ** -17)
    assert abs(by_w - (dw.double() * dwd.double()).sum().item()) <= size * 2.0 ** -15


def test_streams_graphs_and_refusals():
    g = torch.Generator(device=DEV).manual_seed(8)
    q, gq = rows(g, 33, 4, 128, "bf16"), rows(g, 33, 4, 128, "bf16")
    pos, plan = torch.arange(33, dtype=torch.int32, device=DEV), osc.RopePlan(128)
    w = rows(g, 1, 1, 128, "bf16")[0, 0]
    want, dwant = osc.norm_rope(plan, q, None, pos, w)[0], osc.norm_rope_backward(plan, q, None, pos, gq, None, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q)
    osc.norm_rope(plan, q, None, pos, w, q_out=out, stream=s)
    got = osc.norm_rope_backward(plan, q, None, pos, gq, None, w, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(got[0], dwant[0]) and torch.equal(got[2], dwant[2])
    assert (got[3] == 0).all()                                           # no k: its weight's gradient is zero
    graphs, results = [], []
    for _ in range(2):                                                   # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(osc.norm_rope_backward(plan, q, None, pos, gq, None, w))
        graphs.append(graph)
    q.copy_(q.flip(0))
    want = osc.norm_rope_backward(plan, q, None, pos, gq, None, w)
    for graph in graphs:
        graph.replay()
    for r in results:
        assert torch.equal(r[0], want[0]) and torch.equal(r[2], want[2])
    good = dict(plan=plan, q=q, k=None, positions=pos)
    for bad in (dict(q=q.double()), dict(k=q.float()), dict(q_out=out[:, :3]), dict(positions=pos[:32]), dict(layout=2),
                dict(q=q.transpose(1, 2)), dict(q_weight=w.float()), dict(q_weight=w[:64]), dict(eps=0.0),
                dict(plan=plan_of(128, 3)), dict(q_weight=w.cpu())):
        with pytest.raises(osc.OscarError):
            osc.norm_rope(**{**good, **bad})
    grad = dict(good, grad_q=gq, grad_k=None)
    for bad in (dict(grad_q=gq[:, :3]), dict(grad_q=None), dict(grad_k=gq), dict(grad_q=gq.float()), dict(dq=out[:32]),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(osc.OscarError):
            osc.norm_rope_backward(**{**grad, **bad})
    for bad in (pos, pos.repeat(2, 1)):
        with pytest.raises(osc.OscarError):
            osc.rope(plan_of(128, 3), q, None, bad)


def test_nothing_to_do():
    q, plan = torch.zeros(0, 4, 128, device=DEV), osc.RopePlan(128)
    pos = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert osc.norm_rope(plan, q, None, pos)[0].shape == q.shape
    dq, dk, dqw, dkw = osc.norm_rope_backward(plan, q, None, pos, q, None)
    assert dq.shape == q.shape and dk is None and (dqw == 0).all() and (dkw == 0).all()
    assert osc.norm_rope_backward(plan, q, None, pos, q, None, weight_grads=False)[2:] == (None, None)
