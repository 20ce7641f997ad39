"""Reference of the tree attention in 64 bits over a cache's pool bytes, with a bound on the kernel's rounding."""
from __future__ import annotations

import numpy as np

from oracle import pool as P
from oracle.rotation import composite_rotation


def random_mask(rng, B, T, kind):
    """bool [B, T, T]: which drafted nodes a node attends to."""
    i = np.arange(T)
    if kind == "chain":
        return np.tile(i[:, None] >= i, (B, 1, 1))
    if kind == "full":
        return np.ones((B, T, T), bool)
    if kind == "none":
        return np.zeros((B, T, T), bool)
    if kind == "random":                                   # any pattern, some rows empty
        m = rng.random((B, T, T)) < 0.3
        m[:, ::3] = False
        return m
    m = np.zeros((B, T, T), bool)
    for b in range(B):
        for j in range(T):
            p = rng.integers(-1, j) if j else -1
            if p >= 0:
                m[b, j] = m[b, p]
            m[b, j, j] = True
    return m


def mask_words(m):
    B, T, _ = m.shape
    W = -(-T // 64)
    bits = np.zeros((B, T, 64 * W), np.uint8)
    bits[..., :T] = m
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int64)


def attend(pm: P.PoolModel, prm, L, hist_pt, bf16_pt, v_absorbed, q, kd, vd, mask, sm_scale):
    """One request: q [n, Hq, d], kd, vd [n, Hkv, d] float64, mask bool [n, n].

    Returns o [n, Hq, d], lse [n, Hq] and bounds on their errors before the output's rounding. The bound counts, to
    first order, the kernel's roundings. History logits: query row and dequantised key to fp16 (2^-11 relative per
    product each; the rotation's bf16 parts 2^-16 and the float32 sums below 2^-17 more). Weights: to fp16 (2^-11; the
    exponential's 2^-21 and flushed weights below 2^-23 of the row's largest per token are less), drafted and BF16
    weights as two bf16 parts (2^-16). History values to fp16 (2^-11). Codebook and compact scale and zero to fp16
    before the key and value are formed: 2^-11 of |scale code| and of |zero| again; both are bounded by the group's
    range here, 6 times the value's share on average, so the factor 4 below holds for all formats. A relative error e_t
    of the weights moves o by sum p_t e_t (v_t - o)."""
    n, hq, d = q.shape
    hkv = kd.shape[1]
    gq = hq // hkv
    o, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    bound, lse_bound = np.zeros((n, hq, d)), np.zeros((n, hq))
    u = 2.0 ** -11
    for h in range(hkv):
        seg, kk, vv = P.gather_request(pm, L, hist_pt, bf16_pt, heads=[h], params=prm) if L else ([], np.zeros((0, 1, d)),
                                                                                                  np.zeros((0, 1, d)))
        hist = np.array([s == "history" for s in seg], bool)
        rk, rv = (composite_rotation(np.asarray(x, np.float64)) for x in (prm[h].u_k, prm[h].u_v))
        k = np.concatenate([kk[:, 0], kd[:, h]])
        v = np.concatenate([vv[:, 0], vd[:, h]])
        hist = np.concatenate([hist, np.zeros(n, bool)])
        turned = v.copy()
        if not v_absorbed:
            turned[hist] = v[hist] @ rv.T
        # spread of a history value's own rounding, in the output's basis
        spread = np.abs(v) if v_absorbed else np.where(hist[:, None], np.linalg.norm(v, axis=1)[:, None], np.abs(v))
        for i in range(n):
            see = np.concatenate([np.ones(L, bool), mask[i]])
            if not see.any():
                continue
            for e in range(h * gq, (h + 1) * gq):
                x, a = np.empty(len(k)), np.empty(len(k))
                qr = q[i, e] @ rk
                with np.errstate(invalid="ignore", over="ignore"):
                    x[hist], x[~hist] = k[hist] @ qr, k[~hist] @ q[i, e]
                    a[hist], a[~hist] = np.abs(k[hist]) @ np.abs(qr), np.abs(k[~hist]) @ np.abs(q[i, e])
                x, a, w, sp, hh = sm_scale * x[see], sm_scale * a[see], turned[see], spread[see], hist[see]
                m = x.max()
                p = np.exp(x - m)
                s = p.sum()
                p /= s
                o[i, e] = p @ w
                lse[i, e] = m + np.log(s)
                err = np.where(hh, 4 * 2 * u * a, 2.0 ** -17 * a) + 2.0 ** -18
                bound[i, e] = (p * (err + np.where(hh, 2 * u, 2.0 ** -15))) @ np.abs(w - o[i, e]) + \
                    4 * u * ((p * hh) @ sp) + 2.0 ** -18 * (p @ np.abs(w)) + 2.0 ** -30
                lse_bound[i, e] = p @ err + 2.0 ** -18 * (1 + np.abs(lse[i, e]))
    return o, lse, bound, lse_bound


def attend_rounded(pm: P.PoolModel, prm, L, hist_pt, bf16_pt, q, kd, vd, mask, sm_scale, compact=False):
    """One request (fp16 metadata, V absorbed), with the history's operands rounded as the kernel rounds them: the
    rotated query row scaled by a power of two, and every dequantised key and value, to fp16. What is left of the
    kernel's error is its weights' rounding to fp16 and float32 arithmetic. Compact metadata: keys and values are whole
    multiples of half a step of their group's grid and not rounded; the query row is rounded in units of the steps.

    Returns o and the standard deviation of o from the weights' rounding. Rounding a weight p to fp16 makes a relative
    error of at most 2^-11, spread over its interval: a variance of at most 2^-22 / 3, independent from token to token.
    The sum of the weights is not rounded, so o moves by sum p_t e_t v_t: a variance of sum p_t^2 v_t^2 2^-22 / 3. Of
    thousands of terms the sum is close to normal, and 8 deviations are not passed once in 10^15."""
    n, hq, d = q.shape
    gq = hq // kd.shape[1]
    o, dev = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for h in range(kd.shape[1]):
        seg, kk, vv = P.gather_request(pm, L, hist_pt, bf16_pt, heads=[h], params=prm)
        hist = np.array([s == "history" for s in seg] + [False] * n, bool)
        k, v = np.concatenate([kk[:, 0], kd[:, h]]), np.concatenate([vv[:, 0], vd[:, h]])
        unit = np.ones(q.shape[2])
        if compact:                                        # the grids' steps, of the larger one
            unit = np.repeat(prm[h].tau_k.reshape(2, -1).max(1), 64).astype(np.float32)
            unit = unit / unit.max()
        else:
            k[hist], v[hist] = k[hist].astype(np.float16), v[hist].astype(np.float16)
        rk = composite_rotation(np.asarray(prm[h].u_k, np.float64))
        for i in range(n):
            see = np.concatenate([np.ones(L, bool), mask[i]])
            for e in range(h * gq, (h + 1) * gq):
                qr = (q[i, e] @ rk).astype(np.float32)
                scale = 2.0 ** (10 - np.frexp(np.abs(qr).max())[1])
                qr = (qr * (np.float32(scale) * unit)).astype(np.float16).astype(np.float64) / (scale * unit)
                x = np.where(hist, k @ qr, k @ q[i, e])[see] * sm_scale
                p = np.exp(x - x.max())
                p /= p.sum()
                o[i, e] = p @ v[see]
                dev[i, e] = np.sqrt((p * hist[see]) ** 2 @ v[see] ** 2 * 2.0 ** -22 / 3)
    return o, dev
