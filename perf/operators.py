"""The operators of a draft-verification step over the mixed cache, each with its plain form.

A speculative decoder checks a tree of drafted tokens at once: it lays out pages and slots for the
new lengths (``tables``), turns the tree's parents into masks and positions (``layout``), rotates
queries and keys by their positions (``rope``), attends from every drafted node over the committed
cache and the node's drafted ancestors (``tree``) and moves the accepted path into the cache
(``commit``). ``run`` computes one of them, in plain torch operations or, where ``own`` is true,
through the library's public calls.
"""
import math

import numpy as np
import torch

own = False

D, G, P = 128, 64, 64            # head size, quantisation group, tokens per page
SINK, RECENT = 64, 256
NBF = (SINK + RECENT) // P
HEADS = {"8b": (32, 8), "32b": (64, 8), "mha": (8, 8), "pair": (8, 4)}   # (query heads, kv heads)
META = {"f16": 0, "u8": 1, "cb": 2}
CODEBOOK = {"k": (0, 92, 163, 255), "v": (5, 90, 141, 240)}


# ---- cases ---------------------------------------------------------------------------------------------
def listed():
    return [
        # admission of one short prompt: the smallest call, all latency
        dict(name="tables 1 prompt of 777", op="tables", B=1, lo=777, hi=777, grow=0),
        # a batch whose prompts have just arrived, a slot for each of their tokens
        dict(name="tables 64 prompts to 16K", op="tables", B=64, lo=900, hi=16384, grow=0),
        # one request's drafted tree
        dict(name="layout 26 nodes", op="layout", B=1, T=26),
        # a large batch of the widest trees
        dict(name="layout 256 trees of 256", op="layout", B=256, T=256),
        # a verify step of one request far into a long context
        dict(name="rope 5 nodes at 102K", op="rope", N=5, heads="8b", dim=128, rot=128, style="half", dtype="bf16",
             scaling="yarn", inverse=False, top=102400),
        # the gradient of a long prompt's positions, part of the head, neighbouring pairs
        dict(name="rope gradient 49,153 tokens", op="rope", N=49153, heads="8b", dim=128, rot=64, style="pairs",
             dtype="bf16", scaling="linear", inverse=True, top=131072),
        # a chat turn's short chain: latency counts
        dict(name="tree 4 nodes over 1.5K", op="tree", B=1, T=4, heads="8b", lo=1500, hi=1500, meta="f16",
             explicit=False, shape="chain"),
        # an ordinary serving batch, ragged lengths and trees
        dict(name="tree 26 nodes, 8 x 1K-12K", op="tree", B=8, T=26, heads="8b", lo=1000, hi=12000, meta="u8",
             explicit=False, shape="tree"),
        # 64 query heads, explicit value rotation, codebook levels
        dict(name="tree 17 nodes, 64 heads, 33K", op="tree", B=2, T=17, heads="32b", lo=30001, hi=33000, meta="cb",
             explicit=True, shape="tree"),
        # a wide tree over a 102,400-token context: the most arithmetic
        dict(name="tree 64 nodes over 102,400", op="tree", B=1, T=64, heads="8b", lo=102400, hi=102400, meta="f16",
             explicit=False, shape="tree"),
        # one request accepts three tokens
        dict(name="commit 3 of 8", op="commit", B=1, T=8, A=3, heads="8b", lo=1000, hi=1000, explicit=False),
        # a batch accepts ragged paths, values rotated back by the cache
        dict(name="commit 64 x up to 15 of 40", op="commit", B=64, T=40, A=15, heads="8b", lo=100, hi=2000,
             explicit=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "layout", "rope", "tree", "tree", "commit"])
    heads = rng.choice(["8b", "8b", "32b", "mha", "pair"])
    if op == "tables":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 16384)
        return dict(op=op, B=B, lo=max(1, hi // 8), hi=hi, grow=rng.choice([0, 1, 5, 40]))
    if op == "layout":
        return dict(op=op, B=_log(rng, 1, 256), T=_log(rng, 1, 256))
    if op == "rope":
        dim = rng.choice([64, 128, 128, 256])
        most = 49153 * 40 * 64 // (dim * sum(HEADS[heads]))
        return dict(op=op, N=_log(rng, 1, max(2, most)), heads=heads, dim=dim, rot=rng.choice([dim, dim // 2, 24]),
                    style=rng.choice(["half", "pairs"]), dtype=rng.choice(["bf16", "f16", "f32"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), inverse=rng.choice([False, True]),
                    top=_log(rng, 100, 1000000))
    if op == "tree":
        T, B = _log(rng, 1, 200), _log(rng, 1, 16)
        hi = _log(rng, 1, max(2, min(100000, 200_000_000 // (T * B * HEADS[heads][0]), 400_000 // B)))
        return dict(op=op, B=B, T=T, heads=heads, lo=max(0, hi // rng.choice([1, 2, 6]) - 1), hi=hi,
                    meta=rng.choice(["f16", "u8", "cb"]), explicit=rng.choice([False, True]),
                    shape=rng.choice(["chain", "tree"]))
    T = _log(rng, 1, 64)
    hi = _log(rng, 2, 2000)
    return dict(op=op, B=_log(rng, 1, 64), T=T, A=rng.randint(1, min(T, 16)), heads=heads, lo=hi // 2, hi=hi,
                explicit=rng.choice([False, True]))


def _hist(L):
    return max(0, L - SINK - RECENT)


def _pages(L):
    return -(-_hist(L) // P)


def work(c):
    mid = (c["lo"] + c["hi"]) / 2 if "lo" in c else 0
    if c["op"] == "tables":
        new = (c["grow"] or mid) * c["B"]                  # a slot of 16 bytes for each new token
        return {"bytes": 16 * new + c["B"] * (8 + 4 * (mid / P)), "flops": 0}
    if c["op"] == "layout":
        n = c["B"] * c["T"]
        return {"bytes": n * (4 + 4 + 8 * (-(-c["T"] // 64))) + 8 * c["B"], "flops": 0}
    if c["op"] == "rope":
        hq, hkv = HEADS[c["heads"]]
        size = 4 if c["dtype"] == "f32" else 2
        n = c["N"] * (hq + hkv)
        return {"bytes": 2 * n * c["dim"] * size + 4 * c["N"], "flops": 3 * n * c["rot"]}
    hq, hkv = HEADS[c["heads"]]
    if c["op"] == "tree":
        block = 72 if c["meta"] == "u8" else 80            # bytes of one token and kv head, K and V
        hist, bf = _hist(mid), min(mid, SINK + RECENT)
        rows = c["B"] * c["T"] * hq
        nbytes = c["B"] * hkv * (hist * block + bf * 4 * D) + c["B"] * c["T"] * (4 * hq + 4 * hkv) * D
        return {"bytes": nbytes, "flops": 4 * D * rows * (mid + c["T"] / 2)}
    n = c["B"] * (1 + c["A"]) / 2 * hkv                    # accepted rows, K and V of each
    return {"bytes": n * (4 * D * 2 + 4 * D * 2 + 80), "flops": n * 2 * D * D * (2 if c["explicit"] else 1)}


# ---- the cache's bytes: packing, quantising, rotations ---------------------------------------------------
_T = np.arange(P)
V_WORD, V_BIT = (_T >> 1) & 3, 16 * (_T & 1) + 4 * (_T >> 4) + 2 * ((_T >> 3) & 1)
V_ORDER = np.stack([_T[V_WORD == w] for w in range(4)])                # [4 words][16 rows]
V_SLOT = np.arange(D) ^ ((np.arange(D) >> 4) & 7)                      # the 16-byte slot of a channel


def _dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda()


def _u32_bytes(w):
    """int64 values of 32 bits -> their little-endian bytes along the last axis."""
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous().view(torch.uint8)


def _pack_k(codes):
    c = codes.to(torch.uint8).unflatten(-1, (D // 4, 4))
    return c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)


def _pack_v(codes):
    """codes [..., 64, 128] -> bytes [..., 2048]: a channel's 64 codes in four words, slots swizzled."""
    c = codes.to(torch.int64).transpose(-1, -2)[..., _dev(V_ORDER)] << _dev(V_BIT[V_ORDER])
    return _u32_bytes(c.sum(-1)[..., _dev(V_SLOT), :].flatten(-2))


def _quantise(y, tau, meta, cb):
    """Clipped groups of 64 channels -> codes [..., 128] and the metadata bytes [..., 8 or 4]."""
    y = torch.minimum(torch.maximum(y, -tau), tau).unflatten(-1, (2, G))
    mn, mx = y.amin(-1), y.amax(-1)
    if meta == "u8":
        top = tau.unflatten(-1, (2, G)).amax(-1)
        step = (top + top) / 255.0
        a = torch.floor((mn + top) / step).clamp(0, 255)
        b = torch.ceil((mx + top) / step).clamp(0, 255)
        s, z = (b - a) * (step / 3.0), (a.double() * step.double() - top.double()).float()
        raw = torch.stack([a, b], -1).to(torch.uint8)
    else:
        s = (mx - mn if meta == "cb" else (mx - mn) / 3.0).half()
        z = mn.half()
        raw = torch.stack([s, z], -1).contiguous().view(torch.uint8)
        s, z = s.float(), z.float()
    t = (y - z[..., None]) / s[..., None]
    if meta == "cb":
        edges = [(cb[i] + cb[i + 1]) / 510.0 for i in range(3)]
        code = sum((t > torch.tensor(e, dtype=torch.float32)).float() for e in edges)
    else:
        code = torch.round(t).clamp(0, 3)
    code = torch.where(s[..., None] == 0, torch.zeros_like(code), code)
    return code.flatten(-2).to(torch.uint8), raw.flatten(-2)


def _random_pages(g, n, hkv, meta, tau):
    """n INT2 page blocks of Gaussian rows (in the rotated basis), as the write path stores them."""
    parts = []
    for kind in "kv":
        x = torch.randn(n, hkv, P, D, generator=g, device="cuda") * 3.0
        codes, raw = _quantise(x, tau[:, None], meta, CODEBOOK[kind])
        parts.append((_pack_k(codes).flatten(-2) if kind == "k" else _pack_v(codes), raw.flatten(-2)))
        del x, codes
    return torch.cat([parts[0][0], parts[1][0], parts[0][1], parts[1][1]], -1).contiguous()


def _hadamard(n):
    h = np.ones((1, 1))
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return h


def _rotations(rng, hkv, dyadic):
    """R [hkv, 128, 128] float64 and the basis U a cache loads, R = U H P_br.

    dyadic: sign flips and a Hadamard matrix per group, entries +-1/8, so that rotated rows of
    coarse values are exact in any order of summation and every code has one right answer."""
    rev = np.array([int(format(i, "07b")[::-1], 2) for i in range(D)])
    H = _hadamard(D) / math.sqrt(D)
    R, U = [], []
    for _ in range(hkv):
        if dyadic:
            r = np.kron(np.eye(2), _hadamard(G) / 8.0) * rng.choice([-1.0, 1.0], size=(D, 1))
            u = r[:, rev] @ H
        else:
            q, t = np.linalg.qr(rng.standard_normal((D, D)))
            u = (q * np.sign(np.diag(t))).astype(np.float32).astype(np.float64)
            r = (u @ H)[:, rev]
        R.append(r)
        U.append(u.astype(np.float32))
    return np.stack(R), np.stack(U)


def _cache(s, c, n_int2, n_bf16):
    """The library's cache over the same pages."""
    import bit_kv_cache_decode_gb300 as osc
    hq, hkv = HEADS[c["heads"]]
    cache = osc.OscarCache(osc.CacheConfig(
        num_layers=1, num_kv_heads=hkv, num_q_heads=hq, num_int2_pages=n_int2, num_bf16_pages=n_bf16,
        max_batch=c["B"], max_splits=8, v_mode=int(c["explicit"]), meta_format=META[c.get("meta", "f16")]))
    cache.set_rotation(0, s["U_k"], s["U_v"], s["tau"].cpu().numpy(), s["tau"].cpu().numpy())
    if c.get("meta") == "cb":
        cache.set_codebook(0, np.tile(np.uint8(CODEBOOK["k"]), (hkv, 1)), np.tile(np.uint8(CODEBOOK["v"]), (hkv, 1)))
    cache.int2_pages(0).copy_(s["int2"])
    cache.bf16_pages(0).copy_(s["bf16"].view(torch.uint8).reshape(n_bf16, hkv, -1))
    s["cache"], s["int2"] = cache, cache.int2_pages(0)
    s["bf16"] = cache.bf16_pages(0).view(torch.bfloat16).reshape(s["bf16"].shape)


def _lens(rng, c):
    lens = rng.integers(c["lo"], c["hi"] + 1, size=c["B"])
    lens[-1] = c["hi"]
    return lens


def _page_tables(rng, lens, most):
    """Page ids of lengths up to `most`, in tables and pools of one size whatever the lengths are."""
    n = [_pages(int(x)) for x in lens]
    width = _pages(most) + 1                               # one page more each, for what is committed
    total = width * len(n)
    ids, pt, at = rng.permutation(total), np.full((len(n), width), -1, np.int32), 0
    for r, k in enumerate(n):
        pt[r, :k + 1] = ids[at:at + k + 1]
        at += k + 1
    bf = rng.permutation(NBF * len(n)).reshape(len(n), NBF).astype(np.int32)
    return pt, bf, total


def _parents(rng, B, T, shape):
    i = np.arange(T)
    if shape == "chain":
        return np.tile(i - 1, (B, 1)).astype(np.int32)
    # most nodes hang on one of the last few, as beams of drafts do
    back = rng.integers(1, 1 + np.minimum(i + 1, 6), size=(B, T))
    return np.maximum(i - back, -1).astype(np.int32)


def _ancestors(parents):
    """bool [B, T, T] on the host: j is i or above it."""
    B, T = parents.shape
    reach = np.zeros((B, T, T), bool)
    for i in range(T):
        p = parents[:, i]
        reach[:, i] = np.where((p >= 0)[:, None], reach[np.arange(B), np.maximum(p, 0)], False)
        reach[:, i, i] = True
    return reach


def _words(reach):
    B, T, _ = reach.shape
    W = -(-T // 64)
    bits = np.zeros((B, T, 64 * W), np.uint8)
    bits[..., :T] = reach
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int64)


# ---- inputs ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    rng, g = np.random.default_rng(seed), torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "tables":
        new = _lens(rng, c)
        old = new.copy() if c["grow"] else np.zeros_like(new)
        new = new + c["grow"]
        pt, bf, need = _page_tables(rng, new, c["hi"] + c["grow"])
        ids = rng.permutation(4 * need + 64).astype(np.int32)
        for r in range(c["B"]):                            # what is held already; the rest is -1
            pt[r, _pages(int(old[r])):] = -1
            bf[r, int(np.ceil(min(old[r], SINK + RECENT) / P)):] = -1
        s |= dict(old=_dev(old, torch.int32), new=_dev(new, torch.int32), hist=_dev(pt), bf=_dev(bf),
                  free_i=_dev(ids), free_b=_dev(rng.permutation(8 * c["B"] + 8).astype(np.int32)),
                  rings=_dev([int(rng.integers(0, len(ids))), len(ids) - 3 * need, int(rng.integers(0, 8 * c["B"])),
                              6 * c["B"] + 8], torch.int32),
                  rings_out=torch.zeros(4, dtype=torch.int32, device="cuda"), width=pt.shape[1],
                  cu=torch.zeros(c["B"] + 1, dtype=torch.int32, device="cuda"),
                  slots=torch.zeros(c["B"] * (c["grow"] or c["hi"]) + 7, 4, dtype=torch.int32, device="cuda"))
        if own:
            import bit_kv_cache_decode_gb300 as osc
            s["cache"] = osc.OscarCache(osc.CacheConfig(
                num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=len(ids),
                num_bf16_pages=8 * c["B"] + 8, max_batch=c["B"], max_splits=1))
        return s
    if c["op"] == "layout":
        T = c["T"]
        s |= dict(parents=_dev(_parents(rng, c["B"], T, "tree")), lens=_dev(rng.integers(0, 100000, c["B"]), torch.int32),
                  n=_dev(rng.integers(max(1, T // 2), T + 1, c["B"]), torch.int32))
        if own:
            import bit_kv_cache_decode_gb300 as osc
            s["cache"] = osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=1, num_q_heads=1, num_int2_pages=1,
                                                        num_bf16_pages=NBF, max_batch=c["B"], max_splits=1))
        return s
    hq, hkv = HEADS[c["heads"]]
    if c["op"] == "rope":
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[c["dtype"]]
        x = torch.randn(c["N"], hq + hkv, c["dim"], generator=g, device="cuda").to(dt)
        s |= dict(q=x[:, :hq], k=x[:, hq:],                # both in one buffer, as a fused projection leaves them
                  pos=torch.randint(0, c["top"], (c["N"],), generator=g, device="cuda", dtype=torch.int32),
                  q_out=torch.zeros(c["N"], hq, c["dim"], dtype=dt, device="cuda"),
                  k_out=torch.zeros(c["N"], hkv, c["dim"], dtype=dt, device="cuda"))
        freq, scale = _frequencies(c)
        s |= dict(freq=_dev(freq), scale=scale)
        if own:
            import bit_kv_cache_decode_gb300 as osc
            kind = {"none": osc.ROPE_NONE, "linear": osc.ROPE_LINEAR, "yarn": osc.ROPE_YARN}[c["scaling"]]
            s["plan"] = osc.RopePlan(c["rot"], base=1e6, scaling=kind, factor=4.0, original_length=32768)
        return s
    lens = _lens(rng, c)
    pt, bf, total = _page_tables(rng, lens, c["hi"])
    n_bf = bf.size
    s |= dict(lens=_dev(lens, torch.int32), hist=_dev(pt), bf=_dev(bf), host_lens=lens)
    dyadic = c["op"] == "commit"
    Rk, s["U_k"] = _rotations(rng, hkv, dyadic)
    Rv, s["U_v"] = _rotations(rng, hkv, dyadic)
    s |= dict(R_k=_dev(Rk), R_v=_dev(Rv))
    T = c["T"]
    if c["op"] == "tree":
        s["tau"] = _dev(rng.uniform(6.0, 9.0, (hkv, D)), torch.float32)
        s["int2"] = _random_pages(g, total, hkv, c["meta"], s["tau"])
        loud = torch.ones(hkv, 1, D, device="cuda")
        loud.scatter_(2, _dev(np.stack([rng.permutation(D)[:4] for _ in range(hkv)]))[:, None], 16.0)
        kv = torch.randn(n_bf, hkv, 2, P, D, generator=g, device="cuda")
        kv[:, :, 0] *= loud
        s["bf16"] = (kv * torch.tensor([1.0, 3.0], device="cuda")[:, None, None]).bfloat16()
        s["q"] = (torch.randn(c["B"], T, hq, D, generator=g, device="cuda") * 0.5).bfloat16()
        s["kd"] = (torch.randn(c["B"], T, hkv, D, generator=g, device="cuda") * loud[:, 0]).bfloat16()
        s["vd"] = (torch.randn(c["B"], T, hkv, D, generator=g, device="cuda") * 3.0).bfloat16()
        n = rng.integers(max(1, T // 2), T + 1, c["B"])
        n[-1] = T
        s |= dict(n=_dev(n, torch.int32), host_n=n, mask=_dev(_words(_ancestors(_parents(rng, c["B"], T, c["shape"])))),
                  scale=1.0 / math.sqrt(D), out=torch.zeros(c["B"], T, hq, D, dtype=torch.bfloat16, device="cuda"))
        if own:
            _cache(s, c, total, n_bf)
            s["ws"] = torch.empty(s["cache"].tree_workspace_bytes(c["B"], T, pt.shape[1]), dtype=torch.uint8,
                                  device="cuda")
        return s
    # commit: values on a grid of 1/64, see _rotations
    grid = lambda *shape: ((torch.randn(*shape, generator=g, device="cuda") * 64).round().clamp(-255, 255) / 64).bfloat16()  # noqa: E731
    s["tau"] = _dev(rng.integers(16, 24, (hkv, D)) / 8.0, torch.float32)
    s["int2"] = _random_pages(g, total, hkv, "f16", s["tau"])
    s["bf16"], s["kd"], s["vd"] = grid(n_bf, hkv, 2, P, D), grid(c["B"], T, hkv, D), grid(c["B"], T, hkv, D)
    A = c["A"]
    path = np.sort(np.argsort(rng.random((c["B"], T)), axis=1)[:, :A], axis=1)
    n = rng.integers(1, A + 1, c["B"])
    n[-1] = A
    s |= dict(path=_dev(path, torch.int32), n=_dev(n, torch.int32), host_path=path, host_n=n)
    if own:
        _cache(s, c, total, n_bf)
    return s


def _frequencies(c):
    """Angles per position of each pair (float64) and the factor of the rotated values."""
    half = c["rot"] // 2
    freq = 1e6 ** (-np.arange(half) / half)
    if c["scaling"] == "linear":
        return freq / 4.0, 1.0
    if c["scaling"] == "yarn":                             # long waves are stretched by 4, short ones stay
        lo, hi = [half * math.log(32768 / (2 * math.pi * b)) / math.log(1e6) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), 2 * half - 1)
        ramp = np.clip((np.arange(half) - lo) / max(hi - lo, 1e-3), 0, 1)
        return freq / 4.0 * ramp + freq * (1 - ramp), 0.1 * math.log(4.0) + 1.0
    return freq, 1.0


# ---- one pass ------------------------------------------------------------------------------------------------
def run(s):
    return {"tables": _run_tables, "layout": _run_layout, "rope": _run_rope, "tree": _run_tree,
            "commit": _run_commit}[s["case"]["op"]](s)


def _run_tables(s):
    if own:
        s["cache"].build_tables(s["old"], s["new"], s["hist"], s["bf"], s["free_i"], s["free_b"], s["rings"],
                                max_tokens=s["slots"].shape[0], rings_out=s["rings_out"], cu_tokens=s["cu"],
                                slots=s["slots"])
        return {k: s[k] for k in ("hist", "bf", "rings_out", "cu", "slots")}
    old, new = s["old"].long(), s["new"].long()

    def pages(L):                                          # [B], [B]: history pages and BF16 pages of a length
        bf = (L.clamp(max=SINK) + P - 1) // P + ((L - SINK).clamp(0, RECENT) + P - 1) // P
        return ((L - SINK - RECENT).clamp(min=0) + P - 1) // P, bf

    out = []
    for table, held, wanted, ring, at in ((s["hist"], pages(old)[0], pages(new)[0], s["free_i"], 0),
                                          (s["bf"], pages(old)[1], pages(new)[1], s["free_b"], 2)):
        k = torch.arange(table.shape[1], device="cuda")
        fresh = (k >= held[:, None]) & (k < wanted[:, None])
        order = fresh.flatten().cumsum(0).reshape(fresh.shape) - 1
        ids = ring[(s["rings"][at] + order.clamp(min=0)) % ring.numel()]
        table.copy_(torch.where(fresh, ids, table))
        took = (wanted - held).sum()
        out += [(s["rings"][at] + took) % ring.numel(), s["rings"][at + 1] - took]
    s["rings_out"].copy_(torch.stack(out))
    s["cu"][1:] = (new - old).cumsum(0)
    t = torch.arange(s["slots"].shape[0], device="cuda")
    r = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    used, r = r < old.numel(), r.clamp(max=old.numel() - 1)
    pos, L = t - s["cu"].long()[r] + old[r], new[r]
    region = torch.where(pos < SINK, 0, torch.where(pos >= L - RECENT, 2, 1))
    ringpos = (pos - SINK).clamp(min=0) % RECENT
    i = (pos - SINK).clamp(0, s["width"] * P - 1)
    page = torch.where(region == 0, s["bf"].long()[r, (pos // P).clamp(max=NBF - 1)],
                       torch.where(region == 1, s["hist"].long()[r, i // P], s["bf"].long()[r, SINK // P + ringpos // P]))
    row = torch.where(region == 2, ringpos % P, torch.where(region == 1, i % P, pos % P))
    s["slots"].copy_(torch.where(used[:, None], torch.stack([pos, region, page, row], -1).int(), s["slots"]))
    return {k: s[k] for k in ("hist", "bf", "rings_out", "cu", "slots")}


def _run_layout(s):
    if own:
        mask, pos = s["cache"].tree_layout(s["parents"], s["lens"], n_draft=s["n"])
        return {"mask": mask, "positions": pos}
    B, T = s["parents"].shape
    i = torch.arange(T, device="cuda")
    reach = (s["parents"][..., None] == i).float() + torch.eye(T, device="cuda")
    for _ in range((T - 1).bit_length()):                  # ancestors within 1, 2, 4, ... steps
        reach = (reach @ reach).clamp(max=1.0)
    live = i < s["n"][:, None]
    reach = torch.where(live[..., None], reach, 0.0).long()
    pos = torch.where(live, s["lens"][:, None] + reach.sum(-1) - 1, -1).int()
    W = -(-T // 64)
    words = torch.nn.functional.pad(reach, (0, 64 * W - T)).unflatten(-1, (W, 64)) << torch.arange(64, device="cuda")
    return {"mask": words.sum(-1), "positions": pos}


def _run_rope(s):
    c = s["case"]
    if own:
        import bit_kv_cache_decode_gb300 as osc
        osc.rope(s["plan"], s["q"], s["k"], s["pos"], layout=osc.ROPE_HALF if c["style"] == "half" else osc.ROPE_PAIRS,
                 inverse=c["inverse"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    angle = s["pos"].double()[:, None] * s["freq"] * (-1.0 if c["inverse"] else 1.0)
    cos, sin = (angle.cos() * s["scale"]).float()[:, None], (angle.sin() * s["scale"]).float()[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        rot, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["style"] == "half":
            a, b = rot[..., :c["rot"] // 2], rot[..., c["rot"] // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[name] = torch.cat([y, rest], -1).to(s[name].dtype)
    return out


def _unpack(blocks, meta, tau):
    """Dequantised K and V [..., 64, 128] (float32, rotated basis) of page blocks [..., bytes]."""
    two = torch.arange(4, device="cuda", dtype=torch.uint8) * 2
    kc = ((blocks[..., :2048].unflatten(-1, (P, 32))[..., None] >> two) & 3).flatten(-2)
    words = blocks[..., 2048:4096].contiguous().view(torch.int32).unflatten(-1, (D, 4))[..., _dev(V_SLOT), :]
    vc = ((words[..., _dev(V_WORD)] >> _dev(V_BIT, torch.int32)) & 3).transpose(-1, -2)
    out, half = [], (blocks.shape[-1] - 4096) // 2
    for codes, raw, cb in ((kc, blocks[..., 4096:4096 + half], "k"), (vc, blocks[..., 4096 + half:], "v")):
        if meta == "u8":
            ab = raw.unflatten(-1, (P, 2, 2)).float()
            top = tau.unflatten(-1, (2, G)).amax(-1)[..., None, :]                # [hkv, 1, 2]
            step = (top + top) / 255.0
            scale = (ab[..., 1] - ab[..., 0]) * (step / 3.0)
            zero = (ab[..., 0].double() * step.double() - top.double()).float()
        else:
            sz = raw.contiguous().view(torch.float16).unflatten(-1, (P, 2, 2)).float()
            scale, zero = sz[..., 0], sz[..., 1]
        level = codes.float()
        if meta == "cb":
            level = _dev(CODEBOOK[cb], torch.float32)[codes.long()] / 255.0
        out.append((level.unflatten(-1, (2, G)) * scale[..., None] + zero[..., None]).flatten(-2))
    return out


def _run_tree(s):
    c = s["case"]
    if own:
        s["cache"].tree_attention(0, s["q"], s["kd"], s["vd"], s["mask"], s["lens"], s["hist"], s["bf"], s["scale"],
                                  n_draft=s["n"], out=s["out"], workspace=s["ws"])
        return s["out"]
    B, T, hq, _ = s["q"].shape
    hkv = s["kd"].shape[2]
    gq = hq // hkv
    rows = lambda x: x.unflatten(2, (hkv, gq)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, hkv, T gq, 128]  # noqa: E731
    q = rows(s["q"].float())
    L = s["lens"].long()[:, None]
    # history: all pages of the table, those behind the length masked
    k_h, v_h = [x.transpose(1, 2).flatten(2, 3) for x in _unpack(s["int2"][s["hist"].clamp(min=0).long()], c["meta"],
                                                                 s["tau"])]
    R_k, R_v = s["R_k"].float(), s["R_v"].float()
    there_h = torch.arange(k_h.shape[2], device="cuda") < L - SINK - RECENT
    # sink and ring rows
    kv = s["bf16"][s["bf"].long()].float().permute(0, 3, 2, 1, 4, 5).flatten(3, 4)        # [B, 2, hkv, 320, 128]
    i = torch.arange(SINK + RECENT, device="cuda")
    there_b = torch.where(i < SINK, i < L, i - SINK < L - SINK)
    # drafted rows
    kd, vd = [x.float().transpose(1, 2) for x in (s["kd"], s["vd"])]
    j = torch.arange(T, device="cuda")
    sees = ((s["mask"][..., j // 64] >> (j % 64)) & 1).bool() & (j < s["n"].long()[:, None, None])   # [B, T, T]
    sees = sees.repeat_interleave(gq, 1)[:, None]
    logits = torch.cat([(q @ R_k) @ k_h.transpose(-1, -2), q @ kv[:, 0].transpose(-1, -2), q @ kd.transpose(-1, -2)],
                       -1) * s["scale"]
    shape = logits.shape[:-1]
    there = torch.cat([there_h[:, None, None].expand(*shape, -1), there_b[:, None, None].expand(*shape, -1),
                       sees.expand(*shape, -1)], -1)
    logits = logits.masked_fill_(~there, -math.inf)
    del there
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    del logits
    total = p.sum(-1, keepdim=True)
    n_h, n_b = k_h.shape[2], SINK + RECENT
    zero = lambda v, m: v.masked_fill(~m[:, None, :, None], 0.0)    # noqa: E731
    o = p[..., :n_h] @ zero(v_h, there_h)
    if c["explicit"]:
        o = o @ R_v.transpose(-1, -2)
    o = o + p[..., n_h:n_h + n_b] @ zero(kv[:, 1], there_b) + p[..., n_h + n_b:] @ vd
    o = (o / total).unflatten(2, (T, gq)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    live = (j < s["n"].long()[:, None])[..., None, None]
    s["out"].copy_(torch.where(live, o.to(torch.bfloat16), s["out"]))
    return s["out"]


def _run_commit(s):
    if own:
        s["cache"].commit_draft(0, s["kd"], s["vd"], s["lens"], s["n"], s["hist"], s["bf"], path=s["path"])
        return {"int2": s["int2"], "bf16": s["bf16"]}
    B, A = s["path"].shape
    b = torch.arange(B, device="cuda")[:, None].expand(B, A)
    j = torch.arange(A, device="cuda").expand(B, A)
    live = j < s["n"][:, None]
    b, node, pos = b[live], s["path"].long()[live], (s["lens"].long()[:, None] + j)[live]
    hist, bf = s["hist"].long(), s["bf"].long()
    out = pos >= SINK + RECENT                             # these push the oldest recent token out
    ob, old = b[out], pos[out] - RECENT
    slot, h = (old - SINK) % RECENT, old - SINK
    src = s["bf16"][bf[ob, SINK // P + slot // P], :, :, slot % P].float()                # [M, hkv, 2, 128]
    page, row = hist[ob, h // P], h % P
    int2 = s["int2"]
    words = int2[..., 2048:4096].contiguous().view(torch.int32).unflatten(-1, (D, 4)).long() & 0xffffffff
    kraw = int2[..., 4096:4608].unflatten(-1, (P, 8))
    vraw = int2[..., 4608:].unflatten(-1, (P, 8))
    x = (src[:, :, 0].transpose(0, 1) @ s["R_k"].float()).transpose(0, 1)
    codes, raw = _quantise(x, s["tau"], "f16", None)
    int2[..., :2048].unflatten(-1, (P, 32))[page, :, row] = _pack_k(codes)
    kraw[page, :, row] = raw
    y = src[:, :, 1]
    if s["case"]["explicit"]:
        y = (y.transpose(0, 1) @ s["R_v"].float()).transpose(0, 1)
    codes, raw = _quantise(y, s["tau"], "f16", None)
    vraw[page, :, row] = raw
    # each row has bit fields of its own: clear them, then set them
    w, bit = _dev(V_WORD)[row], _dev(V_BIT)[row][:, None, None]
    heads, chan = torch.arange(codes.shape[1], device="cuda")[:, None], _dev(V_SLOT)
    at = (page[:, None, None], heads, chan, w[:, None, None])
    clear, put = torch.zeros_like(words), torch.zeros_like(words)
    clear.index_put_(at, (torch.full_like(codes, 3).long() << bit), accumulate=True)
    put.index_put_(at, codes.long() << bit, accumulate=True)
    int2[..., 2048:4096] = _u32_bytes(((words & ~clear) | put).flatten(-2))
    # the new rows
    slot = (pos - SINK).clamp(min=0) % RECENT
    page = torch.where(pos < SINK, bf[b, (pos // P).clamp(max=NBF - 1)], bf[b, SINK // P + slot // P])
    row = torch.where(pos < SINK, pos % P, slot % P)
    s["bf16"][page, :, :, row] = torch.stack([s["kd"][b, node], s["vd"][b, node]], 2)
    return {"int2": int2, "bf16": s["bf16"]}


# ---- 64 bits -----------------------------------------------------------------------------------------------
def exact(case, seed):
    """Whole-number operators have one right answer and no value here."""
    if case["op"] in ("tables", "layout"):
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](s)


def _exact_rope(s):
    """A pair is a complex number turned by exp(i angle)."""
    c = s["case"]
    turn = torch.polar(torch.full_like(s["freq"], s["scale"]).expand(c["N"], -1).contiguous(),
                       s["pos"].double()[:, None] * s["freq"])[:, None]
    if c["inverse"]:
        turn = turn.conj()
    out = {}
    for name in ("q", "k"):
        y = s[name].double()
        half = c["rot"] // 2
        first = torch.arange(half, device="cuda") * (1 if c["style"] == "half" else 2)
        second = first + (half if c["style"] == "half" else 1)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _levels(blocks, meta, tau, kind):
    """float64 rows [tokens, 128] of one head's page blocks [pages, bytes], each byte's codes looked up."""
    n, half = len(blocks), (blocks.shape[1] - 4096) // 2
    if kind == "k":
        table = np.array([[(x >> (2 * i)) & 3 for i in range(4)] for x in range(256)], np.uint8)
        codes = table[blocks[:, :2048]].reshape(n, P, D)
    else:
        codes = np.empty((n, P, D), np.uint8)
        for c in range(D):
            at = 2048 + 16 * int(V_SLOT[c])
            whole = np.ascontiguousarray(blocks[:, at:at + 16]).view("<u4").astype(np.int64)
            codes[:, :, c] = (whole[:, V_WORD] >> V_BIT) & 3
    raw = np.ascontiguousarray(blocks[:, 4096:4096 + half] if kind == "k" else blocks[:, 4096 + half:])
    if meta == "u8":
        ab = raw.reshape(n, P, 2, 2).astype(np.float64)
        top = tau.reshape(2, G).max(-1).astype(np.float32)
        step = ((top + top) / np.float32(255)).astype(np.float32)
        third = (step / np.float32(3)).astype(np.float64)
        zero = ab[..., 0] * step.astype(np.float64) - top.astype(np.float64)
        scale = (ab[..., 1] - ab[..., 0]) * third
    else:
        sz = raw.view(np.float16).reshape(n, P, 2, 2).astype(np.float64)
        scale, zero = sz[..., 0], sz[..., 1]
    level = np.array(CODEBOOK[kind]) / 255.0 if meta == "cb" else np.arange(4.0)
    return (level[codes] * scale.repeat(G, -1) + zero.repeat(G, -1)).reshape(n * P, D)


def _exact_tree(s):
    """Request by request and head by head: keys and values are turned back into the caller's basis,
    then one ordinary softmax runs over the tokens that a node sees."""
    c = s["case"]
    B, T, hq, _ = s["q"].shape
    hkv = s["kd"].shape[2]
    gq = hq // hkv
    tau, blocks = s["tau"].cpu().numpy(), s["int2"].cpu().numpy()
    pt, bf = s["hist"].cpu().numpy(), s["bf"].cpu().numpy()
    out = torch.zeros(B, T, hq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = int(s["host_lens"][b]), int(s["host_n"][b])
        m = s["mask"][b, :n].cpu().numpy().view(np.uint8)
        sees = _dev(np.unpackbits(m, axis=-1, bitorder="little").reshape(n, -1)[:, :n].astype(bool))
        slots = [p if p < SINK else SINK + (p - SINK) % RECENT
                 for p in list(range(min(L, SINK))) + list(range(max(SINK, L - RECENT), L))]
        for h in range(hkv):
            near = s["bf16"][bf[b].tolist()][:, h].double().transpose(0, 1).flatten(1, 2)[:, slots]    # [2, tokens, 128]
            ks, vs = [near[0], s["kd"][b, :n, h].double()], [near[1], s["vd"][b, :n, h].double()]
            if _hist(L):
                mine = blocks[pt[b, :_pages(L)], h]
                far = [_dev(_levels(mine, c["meta"], tau[h], x)[:_hist(L)]) for x in "kv"]
                ks.insert(0, far[0] @ s["R_k"][h].T)
                vs.insert(0, far[1] @ s["R_v"][h].T if c["explicit"] else far[1])
            k, v = torch.cat(ks), torch.cat(vs)
            for e in range(gq):
                x = (s["q"][b, :n, h * gq + e].double() @ k.T) * s["scale"]
                x[:, k.shape[0] - n:] = torch.where(sees, x[:, k.shape[0] - n:], -math.inf)
                out[b, :n, h * gq + e] = torch.softmax(x, -1) @ v
    return out


def _exact_commit(s):
    """Token by token, as a chain of single appends would do it; the packed bytes are compared whole."""
    bf16 = s["bf16"].double()
    for b, n in enumerate(s["host_n"]):
        for i in range(int(n)):
            pos, node = int(s["host_lens"][b]) + i, int(s["host_path"][b, i])
            slot = pos if pos < SINK else SINK + (pos - SINK) % RECENT
            page = int(s["bf"][b, slot // P])
            bf16[page, :, 0, slot % P] = s["kd"][b, node].double()
            bf16[page, :, 1, slot % P] = s["vd"][b, node].double()
    return {"int2": None, "bf16": bf16}
