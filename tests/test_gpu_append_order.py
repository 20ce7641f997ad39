"""An append or decode step straight after a call that writes page tables or pool rows waits for all of it.

The appends read tables and rows before their programmatic wait, so behind such a call their launch must not be a
programmatic dependent. Seen in captured graphs: the dependency into the append's kernel is then a full one."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

B, HKV, PROGRAMMATIC = 2, 1, 1


class Edge(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


def edges(graph):
    """(from, to, type) of a captured graph's dependencies."""
    cu, g, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetEdges_v2(g, None, None, None, ctypes.byref(n)) == 0
    a, b, e = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (Edge * n.value)()
    assert cu.cuGraphGetEdges_v2(g, a, b, e, ctypes.byref(n)) == 0
    return [(a[i], b[i], e[i].type) for i in range(n.value)]


class Loop:
    def __init__(self):
        self.c = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=HKV, num_q_heads=4, num_int2_pages=16,
                                                num_bf16_pages=10, max_batch=B, max_splits=4), device=DEV)
        eye, tau = np.eye(128, dtype=np.float32)[None], np.full((1, 128), 4, np.float32)
        self.c.set_rotation(0, eye, eye, tau, tau)
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)   # noqa: E731
        g = torch.Generator(device=DEV).manual_seed(3)
        self.hist, self.bf = i32(np.arange(16).reshape(B, 8)), i32(np.arange(10).reshape(B, 5))
        self.fi, self.fb, self.rings = i32(np.arange(16)), i32(np.arange(10)), i32([0, 16, 0, 10])
        self.k, self.v = (torch.randn(700, HKV, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
        self.q = torch.randn(B, 4, 128, generator=g, device=DEV).bfloat16()
        self.kd, self.vd = (torch.randn(B, 4, HKV, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
        self.cu, self.lens, self.n, self.after = i32([0, 300, 700]), i32([300, 400]), i32([4, 3]), i32([304, 403])
        self.rows = [t[:, 0].contiguous() for t in (self.kd, self.vd)]

    def write(self, what):
        c = self.c
        if what == "prefill":
            c.quantize_prefill(0, self.k, self.v, self.cu, self.hist, self.bf)
        elif what == "commit":
            c.commit_draft(0, self.kd, self.vd, self.lens, self.n, self.hist, self.bf)
        else:                                              # nothing grows: the tables stay, the call is the same
            c.build_tables(self.lens, self.lens, self.hist, self.bf, self.fi, self.fb, self.rings)

    def append(self, how):
        if how == "append":
            self.c.append_kv(0, *self.rows, self.after, self.hist, self.bf)
        else:
            self.c.decode_step(0, self.q, *self.rows, self.after, self.hist, self.bf, 0.1)


def chain(graph):
    """The types of the dependencies along the kernels of a graph that is one chain."""
    es = edges(graph)
    nxt = {a: (b, t) for a, b, t in es}
    assert len(nxt) == len(es)
    at = (set(nxt) - {b for _, b, _ in es}).pop()
    out = []
    while at in nxt:
        at, t = nxt[at]
        out.append(t)
    return out


@pytest.mark.parametrize("what", ["prefill", "commit", "tables"])
@pytest.mark.parametrize("how,kernels", [("append", 1), ("step", 3)])
def test_captured(what, how, kernels):
    s = Loop()
    s.write("prefill")
    s.write(what)                                          # what a first call sets up
    s.append(how)
    g = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.write(what)
        s.append(how)
        s.append(how)                                      # behind an append: the overlap is kept
    types = chain(g)
    first = len(types) - 2 * kernels                       # the dependency into the first append
    assert types[first] != PROGRAMMATIC, types
    assert types[first + kernels] == PROGRAMMATIC, types
    assert s.c.get_status() == 0


def test_notes_are_kept_apart_by_capture():
    # the note of an eager write stays for the eager append that follows: a captured one does not take it
    s = Loop()
    s.write("prefill")
    s.append("append")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.write("commit")                                  # noted for the stream itself
    torch.cuda.synchronize()
    for noted in (False, True):
        g = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(g, stream=side):
            if noted:
                s.write("commit")
            s.append("append")
            s.append("append")
        types = chain(g)
        assert len(types) == 1 + noted and types[-1] == PROGRAMMATIC and (not noted or types[0] != PROGRAMMATIC)


@pytest.mark.parametrize("how", ["append", "step"])
def test_results_straight_after(how):
    a, b = Loop(), Loop()
    for s, wait in ((a, False), (b, True)):
        for what in ("prefill", "tables", "commit"):
            s.write(what)
            if wait:
                torch.cuda.synchronize()
        s.append(how)
        torch.cuda.synchronize()
    assert a.c.get_status() == b.c.get_status() == 0
    assert torch.equal(a.c.pool, b.c.pool)


MANY = """
import ctypes, sys
sys.path.insert(0, "tests")
import torch
from test_gpu_append_order import Loop, PROGRAMMATIC, chain
cu, s = ctypes.CDLL("libcuda.so.1"), Loop()
s.write("prefill")
s.append("append")
torch.cuda.synchronize()
def captured():
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        s.append("append")
        s.append("append")
    return chain(g)[-1] == PROGRAMMATIC
assert captured()
for i in range(300):
    h = ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(h), 1) == 0
    with torch.cuda.stream(torch.cuda.ExternalStream(h.value)):
        s.write("tables")
    torch.cuda.synchronize()
    assert captured() == (i < 255), i
assert s.c.get_status() == 0
"""


def test_more_streams_than_are_told_apart():
    # in a process of its own: from then on all its appends wait
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", MANY], capture_output=True, text=True, cwd=root, env={**os.environ, "PYTHONPATH": root})
    assert r.returncode == 0, r.stderr[-800:]
