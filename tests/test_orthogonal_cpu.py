"""The host's check of a rotation against the definition in 64 bits, on both sides of the limit."""
import ctypes

import numpy as np
import pytest

LIMIT = 1e-3


@pytest.fixture(scope="module")
def orthogonal():
    import __graft_entry__
    __graft_entry__.build()
    import bit_kv_cache_decode_gb300 as osc
    f = osc.lib()._ZN5oscar10orthogonalEPKf                 # oscar::orthogonal, see csrc/kernels.cuh
    f.restype, f.argtypes = ctypes.c_bool, [ctypes.c_void_p]

    def call(u):
        held = np.ascontiguousarray(u, np.float32)          # a converted copy lives until the call is over
        return f(held.ctypes.data)
    return call


def rotation(seed):
    return np.linalg.qr(np.random.default_rng(seed).standard_normal((128, 128)))[0].astype(np.float32)


def off(u):
    u = u.astype(np.float64)
    return np.abs(u.T @ u - np.eye(128)).max()


@pytest.mark.parametrize("seed", range(4))
def test_rotations_are(orthogonal, seed):
    assert orthogonal(rotation(seed)) and orthogonal(np.eye(128)) and orthogonal(rotation(seed).T)
    assert orthogonal(rotation(seed)[:, np.random.default_rng(seed).permutation(128)] * -1)


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("how", ["scale", "column", "pair"])
def test_both_sides_of_the_limit(orthogonal, seed, how):
    seen = set()
    for x in np.concatenate([np.linspace(0.97e-3, 1.03e-3, 41), [1e-5, 5e-4, 2e-3, 0.1]]):
        u = rotation(seed).astype(np.float64)
        i, j = 37 + seed, 90 - seed
        if how == "scale":
            u *= np.sqrt(1 + x)                             # the diagonal is 1 + x
        elif how == "column":
            u[:, i] *= np.sqrt(1 - x)
        else:
            u[:, i] += x * u[:, j]                          # one sum beside the diagonal is x
        u = u.astype(np.float32)
        want = off(u) <= LIMIT
        if abs(off(u) - LIMIT) > 1e-12:
            assert orthogonal(u) == want, (x, off(u))
            seen.add(bool(want))
    assert seen == {True, False}


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 3e38, 1e20])
def test_values_that_are_none(orthogonal, value):
    for i, j in ((0, 0), (127, 127), (64, 3), (3, 127)):
        u = rotation(9)
        u[i, j] = value
        assert not orthogonal(u)
    assert not orthogonal(np.full((128, 128), value)) and not orthogonal(np.zeros((128, 128)))
