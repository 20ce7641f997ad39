"""Rotary positions of rows with more heads than a CTA's row numbers times heads fit 32 bits (8 tokens of more than 23,170
heads, or one of more than 65,535): every head turns as it does in a call of its own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


@pytest.mark.parametrize("N,hq,hkv", [(4_867, 20_007, 10_004), (4_867, 30_011, 0), (700, 70_001, 3), (3, 150_001, 0),
                                      (1_217, 65_536, 0)])
@pytest.mark.parametrize("axes", [1, 2])
def test_many_heads(N, hq, hkv, axes):
    g = torch.Generator(device=DEV).manual_seed(hq)
    x = torch.randn(N, hq + hkv, 4, generator=g, device=DEV, dtype=torch.bfloat16)
    pos = torch.randint(0, 10 ** 5, (N,) if axes == 1 else (axes, N), generator=g, device=DEV, dtype=torch.int32)
    pos[..., N // 2] = -1
    plan = osc.RopePlan(4, axes=None if axes == 1 else [0, 1])
    out, want = torch.zeros_like(x), torch.zeros_like(x)
    q, k = x[:, :hq], x[:, hq:] if hkv else None
    osc.rope(plan, q, k, pos, q_out=out[:, :hq], k_out=out[:, hq:] if hkv else None)
    for a in range(0, hq + hkv, 4096):
        osc.rope(plan, x[:, a:a + 4096], None, pos, q_out=want[:, a:a + 4096])
    assert torch.equal(out, want) and (out[N // 2] == 0).all() and (out[-1] != 0).any(-1).all()
