"""The operators around the mixed cache in one attention layer, each with its plain form.

A served layer normalises and rotates its queries and keys (``norm``, in training ``norm gradient``; images and
video have positions with several axes: ``axes``), attends over the prompt (``prompt``) while the cache stores it,
and appends each further token with the norm and the rotation on the way (``append``). ``run`` computes one of
them, in plain torch operations or, where ``own`` is true, through the library's public calls.
"""
import math

import numpy as np
import torch

own = False

D, P = 128, 64                   # the cache's head size and tokens per page
SINK, RECENT = 64, 256
NBF = (SINK + RECENT) // P
HEADS = {"8b": (32, 8), "32b": (64, 8), "mha": (8, 8), "pair": (8, 4)}   # (query heads, kv heads)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------------------
def listed():
    return [
        # decode steps of five requests with pictures: latency counts
        dict(name="axes 5 tokens", op="axes", N=5, heads="8b", dim=128, rot=128, style="half", dtype="bf16",
             order="blocks", inverse=False, top=102400),
        # a long video prompt, axes interleaved over the pairs
        dict(name="axes 40,961 tokens", op="axes", N=40961, heads="8b", dim=128, rot=128, style="half", dtype="bf16",
             order="interleaved", inverse=False, top=32768),
        # one request's next token
        dict(name="norm 1 token", op="norm", N=1, heads="8b", dim=128, rot=128, style="half", dtype="bf16", axes=1,
             top=102400),
        # a long prompt, 64 query heads
        dict(name="norm 32,769 tokens, 64 heads", op="norm", N=32769, heads="32b", dim=128, rot=128, style="half",
             dtype="bf16", axes=1, top=131072),
        # fine-tuning on a short sequence in 32 bits, neighbouring pairs, half of the head rotated
        dict(name="norm gradient 301 tokens", op="grad", N=301, heads="pair", dim=64, rot=32, style="pairs",
             dtype="f32", axes=3, top=4096),
        # fine-tuning on a long sequence
        dict(name="norm gradient 32,769 tokens", op="grad", N=32769, heads="8b", dim=128, rot=128, style="half",
             dtype="bf16", axes=1, top=32769),
        # a chat turn's prompt
        dict(name="prompt 777 tokens", op="prompt", B=1, lo=777, hi=777, heads="8b"),
        # a serving batch of short, ragged prompts
        dict(name="prompt 64 x 1-901", op="prompt", B=64, lo=1, hi=901, heads="8b"),
        # two documents, 64 query heads
        dict(name="prompt 2 x 8K, 64 heads", op="prompt", B=2, lo=8001, hi=8192, heads="32b"),
        # one long document: the most arithmetic
        dict(name="prompt 32,769 tokens", op="prompt", B=1, lo=32769, hi=32769, heads="8b"),
        # one request's next token into its recent window
        dict(name="append 1 request", op="append", B=1, lo=300, hi=300, heads="8b", rot=128, style="half", axes=1),
        # a large batch, some requests still in their sink tokens; positions with three axes
        dict(name="append 256 requests", op="append", B=256, lo=0, hi=319, heads="8b", rot=64, style="pairs", axes=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "norm", "grad", "prompt", "prompt", "append"])
    heads = rng.choice(["8b", "8b", "32b", "mha", "pair"])
    hq, hkv = HEADS[heads]
    style = rng.choice(["half", "pairs"])
    if op == "prompt":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(32769, int(32769 * math.sqrt(32 / (hq * B)))))
        return dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 2, 50])), hi=hi, heads=heads)
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 256), lo=rng.choice([0, 100]), hi=rng.randint(100, SINK + RECENT - 1),
                    heads=heads, rot=rng.choice([D, D // 2, 24]), style=style, axes=rng.choice([1, 1, 3]))
    dim = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "f16", "f32"])
    most = 32769 * 40 * 128 // (dim * (hq + hkv)) // (2 if dtype == "f32" else 1)
    c = dict(op=op, N=_log(rng, 1, most), heads=heads, dim=dim, rot=rng.choice([dim, dim // 2, 24]), style=style,
             dtype=dtype, top=_log(rng, 100, 1000000))
    if op == "axes":
        return c | dict(order=rng.choice(["blocks", "interleaved"]), inverse=rng.choice([False, True]))
    return c | dict(axes=rng.choice([1, 1, 3]))


def work(c):
    hq, hkv = HEADS[c["heads"]]
    if c["op"] == "prompt":
        lo, hi = c["lo"], c["hi"]
        tokens, squares = c["B"] * (lo + hi) / 2, c["B"] * (lo * lo + lo * hi + hi * hi) / 3
        return {"bytes": tokens * 4 * (hq + hkv) * D + 4 * (c["B"] + 1), "flops": 2 * D * hq * (squares + tokens)}
    if c["op"] == "append":
        n = c["B"] * (hq + 2 * hkv)
        return {"bytes": c["B"] * (hq + 2 * hkv) * D * 4 + 4 * c["B"] * (c["axes"] + 2),
                "flops": n * (4 * D + 3 * c["rot"])}
    size = 4 if c["dtype"] == "f32" else 2
    n, axes = c["N"] * (hq + hkv), c.get("axes", 3)
    each = {"axes": 3 * c["rot"], "norm": 4 * c["dim"] + 3 * c["rot"], "grad": 10 * c["dim"] + 3 * c["rot"]}[c["op"]]
    weights = {"axes": 0, "norm": 2 * size, "grad": 2 * size + 8}[c["op"]] * c["dim"]
    return {"bytes": (3 if c["op"] == "grad" else 2) * n * c["dim"] * size + 4 * axes * c["N"] + weights,
            "flops": n * each}


# ---- inputs ------------------------------------------------------------------------------------------------
def _dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda()


def _axes(rot, n, order):
    """The axis of each pair: whole blocks of pairs (a quarter for time, the rest shared), or one pair in turn."""
    half = rot // 2
    if n == 1:
        return np.zeros(half, np.uint8)
    if order == "interleaved":
        return (np.arange(half) % n).astype(np.uint8)
    t, h = half // 4, (half - half // 4 + 1) // 2
    return np.repeat(np.arange(3, dtype=np.uint8), (t, h, half - t - h))


def _positions(g, axes, n, top):
    """Frames in order, rows and columns of a picture within them; with one axis any positions."""
    if axes == 1:
        return torch.randint(0, top, (n,), generator=g, device="cuda", dtype=torch.int32)
    start = torch.randint(0, top, (1,), generator=g, device="cuda")
    i = torch.arange(n, device="cuda")
    side = 24
    return torch.stack([start + i // side ** 2, start + i // side % side, start + i % side]).int()


def _rotary(s, c, g, n, axes, order="blocks"):
    half = c["rot"] // 2
    freq, of = 1e6 ** (-np.arange(half) / half), _axes(c["rot"], axes, order)
    s |= dict(freq=_dev(freq), axis=_dev(of.astype(np.int64)), pos=_positions(g, axes, n, c.get("top", 40000)))
    if own:
        import bit_kv_cache_decode_gb300 as osc
        s["plan"] = osc.RopePlan(c["rot"], base=1e6, axes=None if axes == 1 else of)
        s["layout"] = osc.ROPE_HALF if c["style"] == "half" else osc.ROPE_PAIRS


def prepare(case, seed):
    c = case
    rng, g = np.random.default_rng(seed), torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    hq, hkv = HEADS[c["heads"]]
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")    # noqa: E731
    if c["op"] == "prompt":
        # lengths spread over the range, in another order for another seed
        lens = rng.permutation(np.linspace(c["hi"], c["lo"], c["B"]).astype(int))
        cu = np.concatenate([[0], np.cumsum(lens)])
        n = int(cu[-1])
        # every query leans to the first token of its sequence, as trained heads do
        lean = randn(hkv, D) * 0.25
        x = randn(n, hq + 2 * hkv, D)                      # q, k and v in one buffer, as a fused projection leaves them
        x[:, :hq] += lean.repeat_interleave(hq // hkv, 0)
        x[_dev(cu[:-1]), hq:hq + hkv] += 4 * lean
        x = x.bfloat16()
        s |= dict(q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:], cu=_dev(cu, torch.int32), host_cu=cu,
                  most=int(lens.max()), scale=1.0 / math.sqrt(D),
                  out=torch.zeros(n, hq, D, dtype=torch.bfloat16, device="cuda"))
        if own:
            s["cache"] = _cache(c, 1, NBF)
        return s
    if c["op"] == "append":
        B = c["B"]
        lens = rng.integers(c["lo"], c["hi"] + 1, size=B)
        lens[-1] = c["hi"]
        _rotary(s, c, g, B, c["axes"])
        if c["axes"] == 1:
            s["pos"] = _dev(lens, torch.int32)
        n_bf = NBF * B + 3
        x = randn(B, hq + 2 * hkv, D).bfloat16()
        s |= dict(q=x[:, :hq].contiguous(), k=x[:, hq:hq + hkv].contiguous(), v=x[:, hq + hkv:].contiguous(),
                  qw=(1 + 0.2 * randn(D)).bfloat16(), kw=(1 + 0.2 * randn(D)).bfloat16(),
                  lens=_dev(lens, torch.int32), host_lens=lens,
                  hist=torch.zeros(B, 1, dtype=torch.int32, device="cuda"),
                  bf=_dev(rng.permutation(n_bf)[:NBF * B].reshape(B, NBF).astype(np.int32)),
                  bf16=randn(n_bf, hkv, 2, P, D).bfloat16(), q_out=torch.zeros_like(x[:, :hq]).contiguous())
        if own:
            s["cache"] = _cache(c, 1, n_bf)
            one = np.tile(np.eye(D, dtype=np.float32), (hkv, 1, 1))
            s["cache"].set_rotation(0, one, one, np.full((hkv, D), 9, np.float32), np.full((hkv, D), 9, np.float32))
            pages = s["cache"].bf16_pages(0)
            pages.copy_(s["bf16"].view(torch.uint8).reshape(pages.shape))
            s["bf16"] = pages.view(torch.bfloat16).reshape(s["bf16"].shape)
        return s
    dt, n, dim = TYPES[c["dtype"]], c["N"], c["dim"]
    loud = torch.ones(dim, device="cuda")                  # a few channels are much larger than the others
    loud[_dev(rng.permutation(dim)[:4])] = 8.0
    x = (randn(n, hq + hkv, dim) * loud).to(dt)
    s |= dict(q=x[:, :hq], k=x[:, hq:])
    if c["op"] == "axes":
        _rotary(s, c, g, n, 3, c["order"])
    else:
        _rotary(s, c, g, n, c["axes"])
        s |= dict(qw=(1 + 0.2 * randn(dim)).to(dt), kw=(1 + 0.2 * randn(dim)).to(dt))
    if c["op"] == "grad":
        s |= dict(gq=randn(n, hq, dim).to(dt), gk=randn(n, hkv, dim).to(dt))
    s |= dict(q_out=torch.zeros(n, hq, dim, dtype=dt, device="cuda"), k_out=torch.zeros(n, hkv, dim, dtype=dt, device="cuda"))
    return s


def _cache(c, n_int2, n_bf16):
    import bit_kv_cache_decode_gb300 as osc
    hq, hkv = HEADS[c["heads"]]
    return osc.OscarCache(osc.CacheConfig(num_layers=1, num_kv_heads=hkv, num_q_heads=hq, num_int2_pages=n_int2,
                                          num_bf16_pages=n_bf16, max_batch=c["B"], max_splits=1))


# ---- one pass ------------------------------------------------------------------------------------------------
def run(s):
    return {"axes": _run_axes, "norm": _run_norm, "grad": _run_grad, "prompt": _run_prompt,
            "append": _run_append}[s["case"]["op"]](s)


def _angles(s, sign=1.0):
    """(cos, sin) [N, 1, pairs], the angles in 64 bits."""
    pos = s["pos"].double()
    angle = (pos[:, None] if pos.dim() == 1 else pos[s["axis"]].T) * s["freq"] * sign
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _turn(x, cos, sin, c):
    rot, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["style"] == "half":
        a, b = rot[..., :c["rot"] // 2], rot[..., c["rot"] // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _run_axes(s):
    c = s["case"]
    if own:
        import bit_kv_cache_decode_gb300 as osc
        osc.rope(s["plan"], s["q"], s["k"], s["pos"], layout=s["layout"], inverse=c["inverse"], q_out=s["q_out"],
                 k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cos, sin = _angles(s, -1.0 if c["inverse"] else 1.0)
    return {x: _turn(s[x].float(), cos, sin, c).to(s[x].dtype) for x in ("q", "k")}


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _run_norm(s):
    c = s["case"]
    if own:
        import bit_kv_cache_decode_gb300 as osc
        osc.norm_rope(s["plan"], s["q"], s["k"], s["pos"], s["qw"], s["kw"], eps=EPS, layout=s["layout"],
                      q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cos, sin = _angles(s)
    return {x: _turn(_normed(s[x], s[x + "w"]), cos, sin, c).to(s[x].dtype) for x in ("q", "k")}


def _run_grad(s):
    c = s["case"]
    if own:
        import bit_kv_cache_decode_gb300 as osc
        dq, dk, dqw, dkw = osc.norm_rope_backward(s["plan"], s["q"], s["k"], s["pos"], s["gq"], s["gk"], s["qw"], s["kw"],
                                                  eps=EPS, layout=s["layout"], dq=s["q_out"], dk=s["k_out"])
        return {"q": dq, "k": dk, "qw": dqw, "kw": dkw}
    cos, sin = _angles(s, -1.0)

    def side(x, g, w):
        h, x32 = _turn(g.float(), cos, sin, c), x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
        u, n = h * w.float(), x32 * r
        return ((u - n * (u * n).mean(-1, keepdim=True)) * r).to(x.dtype), (h * n).sum((0, 1), dtype=torch.float64).float()

    (dq, dqw), (dk, dkw) = side(s["q"], s["gq"], s["qw"]), side(s["k"], s["gk"], s["kw"])
    return {"q": dq, "k": dk, "qw": dqw, "kw": dkw}


def _run_prompt(s):
    if own:
        s["cache"].prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["scale"], out=s["out"])
        return s["out"]
    (n, hq, _), hkv, B, L = s["q"].shape, s["k"].shape[1], s["cu"].numel() - 1, s["most"]
    gq = hq // hkv
    # one row of a padded batch for each token; padding reads token 0 and sees itself
    i = torch.arange(L, device="cuda")
    there = i < (s["cu"][1:] - s["cu"][:-1])[:, None]
    at = torch.where(there, s["cu"][:-1].long()[:, None] + i, 0)
    later = i > i[:, None]
    tokens = at[there]
    for h in range(hkv):
        q = s["q"][:, h * gq:(h + 1) * gq].float()[at].transpose(1, 2)        # [B, gq, L, 128]
        k, v = (s[x][:, h].float()[at][:, None] for x in "kv")
        p = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(later, -math.inf)
        p = p.sub_(p.amax(-1, keepdim=True)).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p @ v).div_(total).transpose(1, 2)
        s["out"][tokens, h * gq:(h + 1) * gq] = o[there].to(torch.bfloat16)
        del p, total
    return s["out"]


def _slot(lens):
    return torch.where(lens < SINK, lens, SINK + (lens - SINK) % RECENT)


def _run_append(s):
    c = s["case"]
    if own:
        s["cache"].append_kv_rope(0, s["plan"], s["q"], s["k"], s["v"], s["lens"], s["hist"], s["bf"], q_weight=s["qw"],
                                  k_weight=s["kw"], eps=EPS, positions=None if c["axes"] == 1 else s["pos"],
                                  layout=s["layout"], q_out=s["q_out"])
        return {"q": s["q_out"], "bf16": s["bf16"]}
    cos, sin = _angles(s)
    s["q_out"].copy_(_turn(_normed(s["q"], s["qw"]), cos, sin, c))
    k = _turn(_normed(s["k"], s["kw"]), cos, sin, c).to(torch.bfloat16)
    slot = _slot(s["lens"].long())
    page = s["bf"].long().gather(1, (slot // P)[:, None])[:, 0]
    s["bf16"][page, :, :, slot % P] = torch.stack([k, s["v"]], 2)
    return {"q": s["q_out"], "bf16": s["bf16"]}


# ---- 64 bits -----------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "prompt" and work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    return {"axes": _exact_axes, "norm": _exact_norm, "grad": _exact_grad, "prompt": _exact_prompt,
            "append": _exact_append}[case["op"]](s)


def _pairs(c):
    i = torch.arange(c["rot"] // 2, device="cuda")
    return (i, i + c["rot"] // 2) if c["style"] == "half" else (2 * i, 2 * i + 1)


def _spun(y, s, sign=1.0):
    """A pair is a complex number turned by exp(i angle); y (64 bits) is turned in place."""
    pos = s["pos"].double().reshape(-1, s["pos"].shape[-1])
    angle = torch.zeros(pos.shape[1], len(s["freq"]), dtype=torch.float64, device="cuda")
    for j, f in enumerate(s["freq"].tolist()):
        angle[:, j] = pos[int(s["axis"][j])] * f * sign
    a, b = _pairs(s["case"])
    z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_axes(s):
    sign = -1.0 if s["case"]["inverse"] else 1.0
    return {x: _spun(s[x].double(), s, sign) for x in ("q", "k")}


def _unit(x):
    """Rows of mean square 1 - eps r^2, and 1 / r."""
    rms = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    return x / rms, rms


def _exact_norm(s):
    return {x: _spun(_unit(s[x].double())[0] * s[x + "w"].double(), s) for x in ("q", "k")}


def _exact_grad(s):
    """dx = J^T h with the norm's Jacobian J = (I - n n^T / dim) / rms, n the normed row."""
    out = {}
    for x in ("q", "k"):
        n, rms = _unit(s[x].double())
        h = _spun(s["g" + x].double(), s, -1.0)
        out[x + "w"] = torch.einsum("nhd,nhd->d", h, n)
        u = h * s[x + "w"].double()
        along = torch.einsum("nhd,nhd->nh", n, u) / n.shape[-1]
        out[x] = (u - along[..., None] * n) / rms
    return out


def _exact_prompt(s):
    """Sequence by sequence, head by head, a block of queries at a time over the keys up to its end."""
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    hq, hkv = s["q"].shape[1], s["k"].shape[1]
    for lo, hi in zip(s["host_cu"][:-1].tolist(), s["host_cu"][1:].tolist()):
        for h in range(hkv):
            k, v = s["k"][lo:hi, h].double(), s["v"][lo:hi, h].double()
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for at in range(0, hi - lo, 2048):
                end = min(at + 2048, hi - lo)
                x = torch.einsum("qgd,kd->gqk", s["q"][lo + at:lo + end, mine].double(), k[:end]) * s["scale"]
                seen = torch.ones(end - at, end, dtype=torch.bool, device="cuda").tril(at)
                x = torch.softmax(torch.where(seen, x, -math.inf), -1)
                out[lo + at:lo + end, mine] = torch.einsum("gqk,kd->qgd", x, v[:end])
    return out


def _exact_append(s):
    bf16, q = s["bf16"].double(), _exact_norm(s)
    for b, n in enumerate(s["host_lens"]):
        slot = int(n) if n < SINK else SINK + (int(n) - SINK) % RECENT
        page = int(s["bf"][b, slot // P])
        bf16[page, :, 0, slot % P] = q["k"][b]
        bf16[page, :, 1, slot % P] = s["v"][b].double()
    return {"q": q["q"], "bf16": bf16}
