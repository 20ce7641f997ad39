"""The weights' gradients of norm_rope count every row once, whatever the CTAs' shares.

Rows of 1 and -1 have r = 1, gradients of 1 to 3 in size and quarter turns keep every term h x r of a weight's gradient an integer
other than 0, and so are all partial sums: a float32 sum is exact. (Were r a unit in the last place off, a sum of 150,000 terms of
at most 3 would be off by less than 450,000 x 2^-23 and as much again for 2 units: 0.11.) So a row that is left out or
counted twice shows in every channel."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


def expected(x, g, pos, rot, layout):
    """int64 [D]: sum of h x, h = g turned back by pos quarter turns."""
    x, g = x.long(), g.long()
    i = torch.arange(rot // 2, device=DEV)
    a, b = (i, i + rot // 2) if layout == 0 else (2 * i, 2 * i + 1)
    turns = pos.long()[:, None, None] % 4
    u, v = g[..., a], g[..., b]
    c, s = (turns == 0).long() - (turns == 2).long(), (turns == 1).long() - (turns == 3).long()
    h = g.clone()
    h[..., a], h[..., b] = u * c + v * s, v * c - u * s
    return (h * x)[pos >= 0].sum((0, 1))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 48), (256, 2), (512, 512), (2, 2), (16, 12)])
def test_every_row_counts_once(dim, rot, dtype, layout):
    plan = osc.RopePlan(rot, inv_freq=np.full(rot // 2, np.pi / 2))
    for N, hq, hkv in ((1, 1, 1), (2, 3, 1), (303, 2, 1), (304, 1, 0), (305, 1, 2), (609, 9, 3), (2_433, 32, 8), (9_728, 4, 4),
                       (9_729, 1, 8), (20_011, 4, 1), (70_001, 1, 1)):
        g = torch.Generator(device=DEV).manual_seed(N + dim)
        shift = N % 2                                                    # rows off every boundary too
        # rows and gradients are views of one buffer each, q's heads in front of k's
        def view(values):
            buf = torch.empty(N * (hq + hkv) * dim + 1, dtype=getattr(torch, dtype), device=DEV)
            t = buf[shift:shift + N * (hq + hkv) * dim].view(N, hq + hkv, dim)
            return t.copy_(values)
        sign = lambda: torch.randint(0, 2, (N, hq + hkv, dim), generator=g, device=DEV) * 2 - 1   # noqa: E731
        x = view(sign())
        gr = view(sign() * torch.randint(1, 4, (N, hq + hkv, dim), generator=g, device=DEV))
        pos = torch.randint(0, 8, (N,), generator=g, device=DEV, dtype=torch.int32)
        if N > 2:
            pos[torch.randint(0, N, (max(1, N // 50),), generator=g, device=DEV)] = -1
        k, gk = (x[:, hq:], gr[:, hq:]) if hkv else (None, None)
        _, _, dqw, dkw = osc.norm_rope_backward(plan, x[:, :hq], k, pos, gr[:, :hq], gk, eps=1e-30, layout=layout)
        for dw, s in ((dqw, slice(0, hq)), (dkw, slice(hq, hq + hkv))):
            want = expected(x[:, s], gr[:, s], pos, rot, layout)
            assert ((dw.double() - want).abs() < 0.25).all(), (N, hq, hkv)


@pytest.mark.parametrize("lost", [0, 1])
def test_a_lost_row_would_show(lost):
    g = torch.Generator(device=DEV).manual_seed(1)
    x, gr = (torch.randint(0, 2, (500, 2, 64), generator=g, device=DEV) * 2 - 1 for _ in range(2))
    pos = torch.arange(500, device=DEV, dtype=torch.int32)
    want, keep = expected(x, gr, pos, 64, 0), torch.arange(500, device=DEV) != 321
    other = expected(x[keep], gr[keep], pos[keep], 64, 0) if lost else want
    # a row of two heads adds an even number to a channel; one that adds nothing to all 64 has a chance of 2^-64
    assert bool(((want - other).abs() > 0.25).any()) == bool(lost)
