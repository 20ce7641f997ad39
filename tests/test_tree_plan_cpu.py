"""CPU checks of the host part of the tree attention: how it cuts the pages into slots."""
import ctypes
import subprocess
import sys

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
