"""Rotary positions on the GPU against 64-bit complex rotations.

Tolerance. The rotated value is s (a cos t - b sin t). The table's cosine and sine are float32 results of
sincospif (2 units in the last place at most, 2^-22 absolute) of an angle whose float conversion is off by half a
unit of a value up to 1 half turn (pi 2^-24 2 absolute at most); multiplying by s and forming the two products and
their sum rounds four more times. Together |error| <= s (|a| + |b|) (2^-22 + pi 2^-24 + 4 2^-24) < s (|a| + |b|) 2^-20.5,
and the result is then rounded once to the output type: half a step, eps / 2 relative.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def pairs_of(rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == 0 else (2 * i, 2 * i + 1)


def reference(x, pos, freq, scale, layout, inverse):
    """(rotated float64, error bound) on the CPU."""
    y, rot = x.double().cpu(), 2 * len(freq)
    a, b = pairs_of(rot, layout)
    # pos * f in 80 bits or more, reduced to one turn, so that far positions keep their angle
    turn = np.longdouble(np.asarray(pos, np.int64))[:, None] * (np.longdouble(freq) / (2 * np.longdouble(np.pi)))
    t = torch.from_numpy(np.float64((turn - np.floor(turn)) * 2 * np.longdouble(np.pi)))[:, None]
    t = -t if inverse else t
    u, v = y[..., a].clone(), y[..., b].clone()
    tol = torch.zeros_like(y)
    tol[..., a] = tol[..., b] = scale * (u.abs() + v.abs()) * 2.0 ** -20.5
    y[..., a], y[..., b] = scale * (u * t.cos() - v * t.sin()), scale * (v * t.cos() + u * t.sin())
    live = (torch.as_tensor(np.asarray(pos)) >= 0)[:, None, None]
    return torch.where(live, y, x.double().cpu()), tol


def check(got, x, pos, plan, layout, inverse):
    want, tol = reference(x, pos, plan.inv_freq, plan.scale, layout, inverse)
    eps = torch.finfo(x.dtype).eps / 2
    smallest = torch.finfo(x.dtype).tiny * eps              # half a step of the subnormals
    off = (got.double().cpu() - want).abs()
    bound = tol * (1 + 2 * eps) + want.abs() * eps + smallest
    rot = plan.rotary_dim
    assert torch.equal(got[..., rot:], x[..., rot:])
    assert (off <= bound).all(), (off / bound).max().item()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 24), (64, 20), (256, 256), (96, 2), (80, 80), (512, 512), (34, 6)])
def test_forward_and_inverse(dtype, layout, dim, rot):
    g = torch.Generator(device=DEV).manual_seed(dim + rot)
    N, hq, hkv = 37, 6, 3
    x = torch.randn(N, hq + hkv, dim, generator=g, device=DEV).to(DTYPES[dtype])
    q, k = x[:, :hq], x[:, hq:]
    pos = torch.randint(0, 200_000, (N,), generator=g, device=DEV, dtype=torch.int32)
    pos[:3] = torch.tensor([0, 1, 2 ** 31 - 1])
    plan = osc.RopePlan(rot, base=1e6, scaling=osc.ROPE_YARN, factor=4.0, original_length=32768)
    for inverse in (False, True):
        qo, ko = osc.rope(plan, q, k, pos, layout=layout, inverse=inverse)
        check(qo, q, pos.cpu(), plan, layout, inverse)
        check(ko, k, pos.cpu(), plan, layout, inverse)
    y = x.clone()                                          # in place, both views of one buffer
    osc.rope(plan, y[:, :hq], y[:, hq:], pos, layout=layout, inverse=True, q_out=y[:, :hq], k_out=y[:, hq:])
    assert torch.equal(y[:, :hq], qo) and torch.equal(y[:, hq:], ko)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("shift,token", [(0, 9 * 128), (8, 1160), (1, 1153), (3, 9 * 131)])
def test_strides_and_alignments(layout, shift, token):
    # rows that start on 16 bytes take wide accesses, others single elements
    buf = torch.randn(20 * token + 16, device=DEV).bfloat16()
    head = 131 if token == 9 * 131 else 128
    x = buf.as_strided((20, 9, 128), (token, head, 1), shift)
    pos = torch.arange(20, dtype=torch.int32, device=DEV) * 977
    plan = osc.RopePlan(96, base=10000.0)
    q, _ = osc.rope(plan, x, None, pos, layout=layout)
    check(q, x, pos.cpu(), plan, layout, False)
    t = torch.zeros(9, 20, 128, dtype=torch.bfloat16, device=DEV)      # heads outermost
    osc.rope(plan, x, None, pos, layout=layout, q_out=t.transpose(0, 1))
    assert torch.equal(t.transpose(0, 1), q)


@pytest.mark.parametrize("N", [1, 2, 5, 305, 3000, 20011])
def test_numbers_of_tokens(N):
    g = torch.Generator(device=DEV).manual_seed(N)
    q = torch.randn(N, 2, 64, generator=g, device=DEV)
    pos = torch.randint(0, 10 ** 6, (N,), generator=g, device=DEV, dtype=torch.int32)
    plan = osc.RopePlan(64)
    out, _ = osc.rope(plan, q, None, pos)
    check(out, q, pos.cpu(), plan, 0, False)


def test_padded_rows_stay():
    q = torch.randn(6, 4, 128, device=DEV).bfloat16()
    k = torch.randn(6, 2, 128, device=DEV).bfloat16()
    pos = torch.tensor([5, -1, 7, -1, -1, 0], dtype=torch.int32, device=DEV)
    plan = osc.RopePlan(128)
    qo, ko = torch.full_like(q, -3.0), torch.full_like(k, -3.0)
    osc.rope(plan, q, k, pos, q_out=qo, k_out=ko)
    for i in (1, 3, 4):
        assert (qo[i] == -3).all() and (ko[i] == -3).all()
    live = torch.tensor([0, 2, 5], device=DEV)
    check(qo[live], q[live], pos.cpu()[live.cpu()], plan, 0, False)
    assert torch.equal(qo[5], q[5])                        # position 0: unchanged


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_is_the_gradient(layout):
    # y = rope(x) is linear: <g, (rope(x + e d) - rope(x - e d)) / 2e> = <rope^T g, d> for any d; and rope^T = inverse
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, g, d = (torch.randn(9, 5, 128, generator=gen, device=DEV) for _ in range(3))
    pos = torch.randint(0, 10 ** 5, (9,), generator=gen, device=DEV, dtype=torch.int32)
    plan = osc.RopePlan(64, scaling=osc.ROPE_LINEAR, factor=2.0, scale=1.25)
    f = lambda t: osc.rope(plan, t, None, pos, layout=layout)[0].double()   # noqa: E731
    e = 2.0 ** -3
    lhs = (g.double() * (f(x + e * d) - f(x - e * d)) / (2 * e)).sum()
    rhs = (osc.rope(plan, g, None, pos, layout=layout, inverse=True)[0].double() * d.double()).sum()
    # each of the 9 * 5 * 128 terms is off by at most 2^-20 of values below 2^4, the difference quotient by 2^3 times that
    size = (g.abs().double() * (f(x).abs() + 8)).sum()
    assert abs(lhs - rhs) <= size * 2.0 ** -16
    back = osc.rope(plan, f(x).float(), None, pos, layout=layout, inverse=True)[0]
    want = x.clone()
    want[..., :64] *= 1.25 ** 2                            # the rotation undone, its scale squared
    assert (back - want).abs().max() <= 2.0 ** -18 * 1.6 * 8


def test_other_stream_graph_and_checks():
    q = torch.randn(33, 4, 128, device=DEV).bfloat16()
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    plan = osc.RopePlan(128)
    want, _ = osc.rope(plan, q, None, pos)
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    osc.rope(plan, q, None, pos, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        osc.rope(plan, q, None, pos, q_out=out)
    out.zero_()
    pos += 5
    graph.replay()
    assert torch.equal(out, osc.rope(plan, q, None, pos)[0])
    for bad in (dict(q=q.double()), dict(k=q.float()), dict(q_out=out[:, :3]), dict(positions=pos[:32]),
                dict(q=q.transpose(1, 2)), dict(layout=2)):
        with pytest.raises(osc.OscarError):
            osc.rope(**{**dict(plan=plan, q=q, k=None, positions=pos), **bad})
