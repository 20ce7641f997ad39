"""What loading a layer's rotations leaves in the pool: U and V's transpose, the rotations as the kernels' operands, the
constants, and how long it takes.

The operands hold R = U H P_br in parts. fp16 parts: hi is off by at most 2^-11 |R|, lo by 2^-11 of that or half of fp16's
smallest step, 2^-25. bf16 parts: 2^-8 of what is left, three times (from float32, another 2^-24 of it each time)."""
import ctypes
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")
from oracle.rotation import composite_rotation

D, HKV = 128, 3
FRAG, IMG = 8 * 16 * 32 * 4, 3 * 2 * D * 128 // 4            # words


def inputs(seed, hkv=HKV):
    rng = np.random.default_rng(seed)
    u = [np.stack([np.linalg.qr(rng.standard_normal((D, D)))[0] for _ in range(hkv)]).astype(np.float32) for _ in range(2)]
    return u, rng.uniform(1, 9, (2, hkv, D)).astype(np.float32)


def cache(v_mode, hkv=HKV, layers=2):
    return osc.OscarCache(osc.CacheConfig(num_layers=layers, num_kv_heads=hkv, num_q_heads=hkv, num_int2_pages=1, num_bf16_pages=5,
                                          max_batch=1, max_splits=1, v_mode=v_mode), device=DEV)


def params(c, layer):
    off = [ctypes.c_size_t() for _ in range(3)]
    assert osc.lib().oscar_layer_offsets(c._h, layer, *(ctypes.byref(o) for o in off)) == 0
    n = 3 * D * D + 2 * D + 2 * FRAG + 32 + 2 * IMG
    torch.cuda.synchronize()
    return c.pool[off[2].value:off[2].value + 4 * n * c.cfg.num_kv_heads].cpu().numpy().view(np.float32).reshape(-1, n)


def check_operands(frag, img, R):
    words = frag.view(np.uint32).reshape(8, 16, 32, 4)
    k, n = np.meshgrid(np.arange(D), np.arange(D), indexing="ij")
    lane = (n % 8) * 4 + (k % 8) // 2
    part = [(words[k // 16, n // 8, lane, (k // 8) % 2 + 2 * p] >> (16 * (k % 2))).astype(np.uint16).view(np.float16).astype(np.float64)
            for p in range(2)]
    assert (np.abs(part[0] + part[1] - R) <= 2.0 ** -22 * np.abs(R) + 2.0 ** -25).all()
    assert (np.abs(part[0] - R) <= 2.0 ** -11 * np.abs(R) + 2.0 ** -25).all()
    at = (k // 64) * 16384 + n * 128 + (((k % 64) // 8) ^ (n % 8)) * 16 + (k % 8) * 2
    b = [(img.view(np.uint16)[(at + 32768 * p) // 2].astype(np.uint32) << 16).view(np.float32).astype(np.float64) for p in range(3)]
    for p in range(3):
        assert (np.abs(sum(b[:p + 1]) - R) <= (2.0 ** -8 * (1 + 2.0 ** -15)) ** (p + 1) * np.abs(R) + 2.0 ** -100).all()


@pytest.mark.parametrize("v_mode,with_v", [(0, True), (0, False), (1, True)])
def test_parameters(v_mode, with_v):
    (uk, uv), (tk, tv) = inputs(1)
    c = cache(v_mode)
    c.pool.fill_(0xA5)
    c.set_rotation(1, uk, uv if with_v else None, tk, tv)
    p = params(c, 1)
    o = np.cumsum([0, D * D, D * D, D * D, D, D, FRAG, FRAG, 16, 16, IMG, IMG])
    part = lambda h, i: p[h, o[i]:o[i + 1]]                  # noqa: E731
    for h in range(HKV):
        assert np.array_equal(part(h, 0).reshape(D, D), uk[h])
        assert np.array_equal(part(h, 1).reshape(D, D), uv[h] if with_v else np.zeros((D, D)))
        assert np.array_equal(part(h, 2).reshape(D, D), uv[h].T if with_v else np.zeros((D, D)))
        assert np.array_equal(part(h, 3), tk[h]) and np.array_equal(part(h, 4), tv[h])
        check_operands(part(h, 5), part(h, 9), composite_rotation(uk[h].astype(np.float64)))
        if v_mode:
            check_operands(part(h, 6), part(h, 10), composite_rotation(uv[h].astype(np.float64)))
        else:
            assert not part(h, 6).any() and not part(h, 10).any()
        grid = part(h, 7).reshape(2, 2, 4)
        for kind, t in enumerate((tk[h], tv[h])):
            top = t.reshape(2, 64).max(1)
            step = (top + top) / np.float32(255)
            assert np.array_equal(grid[kind, :, 0], top) and np.array_equal(grid[kind, :, 1], step)
            assert np.array_equal(grid[kind, :, 2], step / np.float32(3))
        assert np.array_equal(part(h, 8).reshape(2, 8)[:, :4], np.tile(np.float32([0, 85, 170, 255]), (2, 1)))
    off0 = c.pool[:c.pool.numel() // 2]
    assert (off0 == 0xA5).all()                              # the other layer stays


def test_a_rotation_that_is_not_orthogonal_changes_nothing():
    (uk, uv), (tk, tv) = inputs(2)
    c = cache(1)
    c.set_rotation(0, uk, uv, tk, tv)
    before = c.pool.clone()
    for which in range(2):
        for h, i, j, x in ((0, 0, 0, 0.01), (HKV - 1, 127, 127, -0.01), (1, 5, 70, np.nan), (2, 70, 5, np.inf)):
            u = [uk.copy(), uv.copy()]
            u[which][h, i, j] += x
            with pytest.raises(osc.OscarError) as e:
                c.set_rotation(0, *u, tk, tv)
            assert e.value.code == osc.ERR_NOT_ORTHOGONAL
    assert torch.equal(c.pool, before)


def test_attention_straight_after_loading():
    # the kernels read parameters before they wait for a kernel before them: what loads them ends with copies
    (u, v), (tk, tv) = inputs(3)
    q = torch.randn(1, 2, HKV, D, device=DEV).bfloat16()
    kv = torch.randn(1, 2, HKV, D, device=DEV).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    args = (q, kv, kv, torch.ones(1, 2, 1, dtype=torch.int64, device=DEV), i32([400]), i32([[0, 0]]), i32([[0, 1, 2, 3, 4]]), 0.1)
    c = cache(1)
    c.pool[:c.int2_pages(0).numel()].random_(0, 60)
    outs = []
    for first, wait in ((u, True), (v, False), (v, True)):
        c.set_rotation(0, first, v, tk, tv)
        if wait:
            torch.cuda.synchronize()
        outs.append(c.tree_attention(0, *args))
    assert torch.equal(outs[1], outs[2]) and not torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("v_mode", [0, 1])
def test_time_of_a_layer(v_mode):
    # 0.5 and 0.6 ms for 8 heads; loops on one host thread took 25 and 40
    (uk, uv), (tk, tv) = inputs(4, 8)
    c = cache(v_mode, 8, 1)
    took = []
    for _ in range(8):
        t = time.perf_counter()
        c.set_rotation(0, uk, uv, tk, tv)
        torch.cuda.synchronize()
        took.append(time.perf_counter() - t)
    assert min(took) < 0.01


@pytest.mark.parametrize("pinned", [False, True])
def test_the_sources_may_change_once_the_call_returns(pinned):
    (uk, uv), (tk, tv) = inputs(5, 8)
    c, busy = cache(1, 8, 1), torch.zeros(1 << 28, device=DEV)
    c.set_rotation(0, uk, uv, tk, tv)
    want = params(c, 0).copy()
    for _ in range(5):
        src = [torch.from_numpy(np.array(x)) for x in (uk, uv, tk, tv)]
        if pinned:
            src = [x.pin_memory() for x in src]
        c.pool.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            busy.add_(1.0)                                 # the copies wait on the stream
        c.set_rotation(0, *(x.numpy() for x in src))
        for x in src:
            x.fill_(7.0)
        assert np.array_equal(params(c, 0).view(np.uint32), want.view(np.uint32))
