"""Rotations of a part of a head: calls that L2 holds and calls that it does not, rows of a power of two of bytes and others give
the same bits, token by token; rows off every boundary stay within the bound of layer_cases.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import layer_cases as L  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dim,rot", [(160, 80), (80, 32), (96, 24), (256, 64), (128, 64), (64, 24), (512, 16), (96, 90)])
def test_long_calls_and_short_ones(dim, rot, dtype, layout):
    N, H = 2 ** 27 // (2 * 40 * dim * 2) + 19, 40                        # more than 2^27 bytes of input and output
    g = torch.Generator(device=DEV).manual_seed(dim + rot)
    x = torch.randn(N, H, dim, generator=g, device=DEV).to(getattr(torch, dtype))
    pos = torch.randint(0, 10 ** 6, (N,), generator=g, device=DEV, dtype=torch.int32)
    plan = osc.RopePlan(rot, base=1e6, scale=1.25)
    for inverse in (False, True):
        q, k = osc.rope(plan, x[:, :33], x[:, 33:], pos, layout=layout, inverse=inverse)
        got = torch.cat([q, k], 1)
        want = torch.cat([osc.rope(plan, x[a:a + 500], None, pos[a:a + 500], layout=layout, inverse=inverse)[0]
                          for a in range(0, N, 500)])
        assert torch.equal(got, want)
        odd = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(N, H, dim).copy_(x)
        got = osc.rope(plan, odd, None, pos, layout=layout, inverse=inverse, q_out=odd)[0]
        # Not the same bits: in u c - v s one product is fused with the difference, and which one is each kernel's own choice.
        # Either is off by the two roundings that the bound counts before the rounding at the end.
        some = torch.cat([torch.arange(0, N, 97), torch.tensor([N - 1])]).to(DEV)
        exact, size = L.turned(x[some].double().cpu(), plan, pos[some].cpu(), layout, inverse)
        L.near(got[some], exact, L.rounded(exact, size * 2.0 ** -20.5, x.dtype))
