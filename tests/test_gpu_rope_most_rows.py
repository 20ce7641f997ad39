"""Rotary positions of as many rows as the call can name: 2^31 - 1, and one more, which is refused."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


def test_two_billion_rows():
    most = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("needs 18 GB")
    pos = torch.zeros(most + 1, dtype=torch.int32, device=DEV)
    x = torch.ones(most + 1, 1, 2, dtype=torch.bfloat16, device=DEV)
    plan = osc.RopePlan(2, base=10000.0)
    at = torch.tensor([0, 5, 2 ** 30, most - 1, most], device=DEV)
    pos[at] = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(osc.OscarError):
        osc.rope(plan, x, None, pos, q_out=x)
    osc.rope(plan, x[:most], None, pos[:most], q_out=x[:most])
    small = torch.ones(4, 1, 2, dtype=torch.bfloat16, device=DEV)
    want, _ = osc.rope(plan, small, None, torch.arange(4, dtype=torch.int32, device=DEV))
    assert torch.equal(x[at[:4]], want) and (x[most] == 1).all()
    assert (x[1:5] == 1).all() and (x[most - 9:most - 1] == 1).all()
