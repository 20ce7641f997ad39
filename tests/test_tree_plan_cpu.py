"""CPU checks of the host part of the tree attention: how it cuts the pages into slots."""
import ctypes
import subprocess
import sys
import time

import pytest

SYMBOL = "_ZN5oscar11tree_splitsEiiiiiiiiPiS0_S0_"          # oscar::tree_splits, see csrc/kernels.cuh


@pytest.fixture(scope="module")
def splits():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_decode_gb300 as osc
    f = getattr(osc.lib(), SYMBOL)
    f.restype = None

    def call(B, T, hkv, gq, nbf, pages, sms=152, max_slots=1 << 20):
        out = [ctypes.c_int(-1) for _ in range(3)]
        f(B, T, hkv, gq, nbf, pages, sms, max_slots, *(ctypes.byref(x) for x in out))
        return tuple(x.value for x in out)                   # history slots, BF16 and draft slots, pages of a slot
    return call


def test_an_empty_batch_has_a_plan():
    # in a process of its own: a division by zero ends the process
    code = ("import ctypes, bit_kv_cache_decode_gb300 as o\n"
            "x = [ctypes.c_int(-1) for _ in range(3)]\n"
            f"o.lib().{SYMBOL}(0, 5, 8, 4, 5, 100, 152, 1 << 20, *(ctypes.byref(v) for v in x))\n"
            "assert x[0].value >= 1 and x[1].value >= 1, [v.value for v in x]\n")
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=__graft_entry__.ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


@pytest.mark.parametrize("B,T,hkv,gq", [(1, 5, 8, 4), (64, 5, 8, 4), (64, 26, 8, 4), (304, 17, 1, 8), (608, 1, 1, 8), (16, 256, 8, 8)])
@pytest.mark.parametrize("pages", [1, 511, 513, 2048, 4097, 16384, 200_000])
@pytest.mark.parametrize("nbf", [5, 129, 2040])
def test_an_accumulator_takes_1024_products(splits, B, T, hkv, gq, pages, nbf):
    streams = 1 if T * gq > 128 else 2
    near = nbf + -(-T // 64)
    s, m, pps = splits(B, T, hkv, gq, nbf, pages)
    assert s * pps >= pages and pps <= streams * 256 and -(-near // m) <= streams * 128
    for slots in (s + m, s + m - 1, 40, 3, 2):               # less workspace: as many as there are, and no refusal
        least = -(-pages // 4096)
        s2, m2, p2 = splits(B, T, hkv, gq, nbf, pages, max_slots=slots)
        assert (s2 == 0) == (least + 1 > slots)
        if s2:
            assert s2 + m2 <= slots and s2 * p2 >= pages and p2 <= 4096


def searched(B, T, hkv, gq, nbf, pages, sms, max_slots):
    """The plan of least cost among all counts of slots, and of equal ones the first."""
    up = lambda n, x: -(-n // x)                             # noqa: E731
    tiles, wide = up(T * gq, 128), T * gq > 128
    streams = 1 if wide else 2
    units = max(1, B * hkv * (up(tiles, 2) if wide else tiles))
    near, pages = nbf + up(T, 64), max(1, pages)
    exact_s, exact_m = up(pages, streams * 256), up(near, streams * 128)
    least_s = min(exact_s, max(up(pages, 4096), max_slots - exact_m))
    least_m = min(exact_m, max(1, max_slots - least_s))
    most_s = max(least_s, min(pages, 2 * sms, 4 * sms // units + 1))
    best = (0.0, 0, 0, 1)
    for m in range(least_m, near + 1):
        if m >= max_slots:
            break
        for s in range(least_s, min(most_s, max_slots - m) + 1):
            h, g = up(pages, s) + 20.0, 5.0 * up(near, m) + 20.0
            more = [0.0 if units * (f * s + m) <= sms else units * (f * s * h + m * g) / sms for f in (1.0, 0.75)]
            cost = max(h, g) + (0.35 * more[0] + (1.0 - 0.35) * more[1] if B > 1 else more[0]) + 0.1 * (s + m)
            if best[0] == 0.0 or cost < best[0]:
                best = (cost, s, m, up(pages, s))
    return best[1:]


@pytest.mark.parametrize("B,T,hkv,gq", [(1, 1, 1, 1), (1, 5, 8, 4), (2, 17, 8, 8), (8, 26, 8, 4), (64, 5, 8, 4), (5, 60, 8, 4)])
@pytest.mark.parametrize("pages", [0, 1, 2, 63, 190, 500, 1595])
@pytest.mark.parametrize("nbf", [5, 20, 67])
@pytest.mark.parametrize("max_slots", [1 << 20, 23, 7, 2])
def test_the_search_finds_the_least_cost(splits, B, T, hkv, gq, pages, nbf, max_slots):
    assert splits(B, T, hkv, gq, nbf, pages, 152, max_slots) == searched(B, T, hkv, gq, nbf, pages, 152, max_slots)


def test_the_search_is_short_whatever_the_window(splits):
    for nbf in (5, 67, 2040):
        took = []
        for _ in range(5):
            t = time.perf_counter()
            for _ in range(20):
                splits(1, 5, 1, 1, nbf, 1600)
            took.append((time.perf_counter() - t) / 20)
        assert min(took) < 2e-4, (nbf, min(took))            # 2.5 ms with every count of slots
