"""Page tables, slots, tree masks and positions built on the GPU, against plain Python."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")

SINK, RECENT, P = 64, 256, 64


def hist_pages(L):
    return -(-max(0, L - SINK - RECENT) // P)


def bf16_pages(L):
    return -(-min(L, SINK) // P) + -(-min(max(L - SINK, 0), RECENT) // P)


class Model:
    """The state a serving loop keeps, and what a call does to it."""

    def __init__(self, B, n_int2, n_bf16, width, seed=0):
        rng = np.random.default_rng(seed)
        self.hist, self.bf = np.full((B, width), -1, np.int32), np.full((B, 5), -1, np.int32)
        self.free = [rng.permutation(n_int2).astype(np.int32), rng.permutation(n_bf16).astype(np.int32)]
        self.rings = [int(rng.integers(n_int2)), n_int2, int(rng.integers(n_bf16)), n_bf16]
        self.lens = np.zeros(B, np.int64)

    def call(self, new):
        tables, counts = (self.hist, self.bf), (hist_pages, bf16_pages)
        slots, cu = [], [0]
        for e in range(2):
            ring, (head, count), cap = self.free[e], self.rings[2 * e:2 * e + 2], len(self.free[e])
            pops, pushes = 0, []
            for r, (o, n) in enumerate(zip(self.lens, new)):
                held, want = counts[e](int(o)), counts[e](int(n))
                if n >= o:
                    for j in range(held, want):
                        tables[e][r, j] = ring[(head + pops) % cap]
                        pops += 1
                else:
                    pushes += [int(x) for x in tables[e][r, :held]]
                    tables[e][r, :held] = -1
            for i, x in enumerate(pushes):
                ring[(head + count + i) % cap] = x
            self.rings[2 * e:2 * e + 2] = [(head + pops) % cap, count - pops + len(pushes)]
        for r, (o, n) in enumerate(zip(self.lens, new)):
            for pos in range(int(o), int(n)):
                if pos < SINK:
                    slots.append((pos, 0, self.bf[r, pos // P], pos % P))
                elif pos >= n - RECENT:
                    at = (pos - SINK) % RECENT
                    slots.append((pos, 2, self.bf[r, 1 + at // P], at % P))
                else:
                    slots.append((pos, 1, self.hist[r, (pos - SINK) // P], (pos - SINK) % P))
            cu.append(len(slots))
        self.lens = np.asarray(new, np.int64)
        return np.array(slots, np.int32).reshape(-1, 4), np.array(cu, np.int32)


def cache_for(m, B=1):
    return osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=len(m.free[0]),
                                          num_bf16_pages=len(m.free[1]), max_batch=B, max_splits=1), device=DEV)


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=DEV)


class Device:
    def __init__(self, m):
        self.hist, self.bf, self.fi, self.fb, self.rings = (dev(x) for x in (m.hist, m.bf, m.free[0], m.free[1], m.rings))

    def same(self, m):
        for a, b in ((self.hist, m.hist), (self.bf, m.bf), (self.fi, m.free[0]), (self.fb, m.free[1]),
                     (self.rings, np.array(m.rings))):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("B,steps", [(1, 6), (3, 8), (37, 6), (300, 4)])
def test_growing_and_released_requests(B, steps):
    rng = np.random.default_rng(B)
    m = Model(B, n_int2=14 * B + 3, n_bf16=5 * B + 1, width=15, seed=B)
    cache, d = cache_for(m), Device(m)
    for step in range(steps):
        new = m.lens + rng.choice([0, 1, 2, 17, 63, 64, 65, 130], size=B)
        if step == 0:
            new = rng.choice([1, 63, 64, 65, 200, 319, 320, 321, 384, 385, 700], size=B)
        elif step > 1:                                     # some finish, some of those start again later
            new[rng.random(B) < 0.3] = 0
        new = np.minimum(new, SINK + RECENT + 14 * P)
        new[(new < m.lens) & (new != 0)] = 0
        old = m.lens.copy()
        slots, cu = m.call(new)
        out = torch.full((len(slots) + 3, 4), -7, dtype=torch.int32, device=DEV)
        _, got_cu, got = cache.build_tables(dev(old), dev(new), d.hist, d.bf, d.fi, d.fb, d.rings, slots=out)
        d.same(m)
        assert np.array_equal(got_cu.cpu().numpy(), cu)
        assert np.array_equal(got[:len(slots)].cpu().numpy(), slots)
        assert (got[len(slots):] == -7).all()              # rows behind the last token stay
    assert cache.get_status() == 0


def test_one_long_prompt_over_many_ctas():
    L = 130_001
    m = Model(1, hist_pages(L) + 2, 5, hist_pages(L))
    cache, d = cache_for(m), Device(m)
    slots, cu = m.call([L])
    rings = torch.zeros(4, dtype=torch.int32, device=DEV)
    before = d.rings.clone()
    for _ in range(3):                                     # rings_out apart: the same call gives the same again
        r, got_cu, got = cache.build_tables([0], [L], d.hist, d.bf, d.fi, d.fb, d.rings, max_tokens=L, rings_out=rings)
        assert torch.equal(d.rings, before) and r is rings
        assert np.array_equal(got.cpu().numpy(), slots) and np.array_equal(got_cu.cpu().numpy(), cu)
        assert rings.tolist() == m.rings
    d.rings = rings
    d.same(m)
    assert cache.get_status() == 0


def test_without_slots_and_empty_batch():
    m = Model(4, 20, 20, 8)
    cache, d = cache_for(m), Device(m)
    m.call([500, 0, 64, 700])
    cache.build_tables([0] * 4, [500, 0, 64, 700], d.hist, d.bf, d.fi, d.fb, d.rings)
    d.same(m)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    cache.build_tables(e, e, torch.zeros(0, 8, dtype=torch.int32, device=DEV), e, d.fi, d.fb, d.rings)
    d.same(m)
    assert cache.get_status() == 0


@pytest.mark.parametrize("old,new,status", [
    ([0, 0], [100, -1], 2), ([-5, 0], [100, 1], 2), ([0, 200], [10, 100], 2),      # negative, shrinking to other than 0
    ([0, 0], [SINK + RECENT + 4 * P + 1, 1], 2),                                   # beyond its page table
    ([0, 0], [600, 600], 32),                                                      # 10 pages of 9
    ([0, 0], [1000, 1], 2),
])
def test_refused_calls_change_nothing(old, new, status):
    m = Model(2, 9, 10, 4)
    if status == 32:
        m = Model(2, 9, 10, 5)
    cache, d = cache_for(m), Device(m)
    slots = torch.full((4000, 4), -7, dtype=torch.int32, device=DEV)
    cu = torch.full((3,), -7, dtype=torch.int32, device=DEV)
    cache.build_tables(old, new, d.hist, d.bf, d.fi, d.fb, d.rings, slots=slots, cu_tokens=cu)
    d.same(m)
    assert (slots == -7).all() and (cu == -7).all()
    assert cache.get_status() == status


def test_too_few_slots_or_a_bad_ring_change_nothing():
    m = Model(2, 30, 10, 8)
    cache, d = cache_for(m), Device(m)
    slots = torch.full((199, 4), -7, dtype=torch.int32, device=DEV)
    cache.build_tables([0, 0], [100, 100], d.hist, d.bf, d.fi, d.fb, d.rings, slots=slots)
    d.same(m)
    assert cache.get_status() == osc.STATUS_BAD_SEQLEN
    for bad in ([-1, 5, 0, 5], [30, 5, 0, 5], [0, 31, 0, 5], [0, 5, 0, -1], [0, 5, 10, 1]):
        rings = dev(bad)
        cache.build_tables([0, 0], [1, 1], d.hist, d.bf, d.fi, d.fb, rings)
        assert rings.tolist() == bad and cache.get_status() == osc.STATUS_BAD_PAGE
    # releasing more than the ring can take back
    cache.build_tables([64, 0], [0, 0], d.hist, d.bf, d.fi, d.fb, d.rings)
    d.same(m)
    assert cache.get_status() == osc.STATUS_BAD_PAGE


def test_table_argument_checks():
    m = Model(2, 9, 10, 4)
    cache, d = cache_for(m), Device(m)
    with pytest.raises(osc.OscarError):
        cache.build_tables([0, 0], [1], d.hist, d.bf, d.fi, d.fb, d.rings)
    with pytest.raises(osc.OscarError):
        cache.build_tables([0, 0], [1, 1], d.hist, d.bf, d.fi[:8], d.fb, d.rings)
    with pytest.raises(osc.OscarError):
        cache.build_tables([0, 0], [1, 1], d.hist, d.bf.long(), d.fi, d.fb, d.rings)
    big = torch.zeros(4097, dtype=torch.int32, device=DEV)
    with pytest.raises(osc.OscarError) as e:
        cache.build_tables(big, big, torch.zeros(4097, 1, dtype=torch.int32, device=DEV), big.repeat(5), d.fi, d.fb, d.rings)
    assert e.value.code == osc.ERR_UNSUPPORTED


# ---- trees -----------------------------------------------------------------------------------------------
def tree_model(parents, n, lens):
    B, T = parents.shape
    W = -(-T // 64)
    mask, pos = np.zeros((B, T, W), np.uint64), np.full((B, T), -1, np.int32)
    for b in range(B):
        sets = []
        for i in range(T):
            p = parents[b, i]
            s = None
            if i < n[b] and p < i and p >= -1:
                s = {i} if p == -1 else (sets[p] | {i} if sets[p] is not None else None)
            sets.append(s)
            if s is not None:
                for j in s:
                    mask[b, i, j // 64] |= np.uint64(1 << (j % 64))
                pos[b, i] = lens[b] + len(s) - 1
    return mask.view(np.int64), pos


def random_parents(rng, B, T, kind):
    i = np.arange(T)
    if kind == "chain":
        return np.tile(i - 1, (B, 1)).astype(np.int32)
    if kind == "star":
        return np.full((B, T), -1, np.int32)
    return np.stack([rng.integers(-1, np.maximum(i, 0)) if T > 1 else np.array([-1]) for _ in range(B)]).astype(np.int32)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 128, 200, 256])
@pytest.mark.parametrize("kind", ["chain", "star", "random"])
def test_tree_layout(T, kind):
    rng = np.random.default_rng(T)
    B = 5
    parents = random_parents(rng, B, T, kind)
    n = rng.integers(0, T + 1, B).astype(np.int32)
    n[0] = T
    lens = rng.integers(0, 2 ** 30, B).astype(np.int32)
    lens[1] = 0
    cache = cache_for(Model(1, 1, 5, 1))
    for nd, ns in ((None, np.full(B, T)), (n, n)):
        mask, pos = cache.tree_layout(parents, lens, n_draft=nd)
        want = tree_model(parents, ns, lens)
        assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])
    assert cache.get_status() == 0


def test_bad_parents_and_counts():
    cache = cache_for(Model(1, 1, 5, 1))
    parents = np.array([[-1, 0, 2, 1, 2, 3, -2, 6, 0, 99]], np.int32)   # nodes 2, 6, 9 are bad; 4 and 7 below them
    mask, pos = cache.tree_layout(parents, [10])
    want = tree_model(parents, [10], [10])
    assert np.array_equal(mask.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[1])
    assert pos.cpu().numpy().tolist() == [[10, 11, -1, 12, -1, 13, -1, -1, 11, -1]]
    assert cache.get_status() == osc.STATUS_BAD_TREE
    for n, live in ((-1, 0), (11, 10)):                    # a count out of range is clamped and reported
        good = np.array([[-1] + list(range(9))], np.int32)
        _, pos = cache.tree_layout(good, [10], n_draft=[n])
        assert (pos.cpu().numpy() >= 0).sum() == live
        assert cache.get_status() == osc.STATUS_BAD_TREE
    with pytest.raises(osc.OscarError) as e:
        cache.tree_layout(np.full((1, 257), -1, np.int32), [1])
    assert e.value.code == osc.ERR_UNSUPPORTED
    with pytest.raises(osc.OscarError):
        cache.tree_layout(good, [1, 2])
    with pytest.raises(osc.OscarError):
        cache.tree_layout(good, [1], mask=torch.zeros(1, 10, 2, dtype=torch.int64, device=DEV))
