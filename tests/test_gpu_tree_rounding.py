"""Tree attention against a reference that rounds the history's operands as the kernel does, in every metadata format and
with V absorbed or rotated: what is left is the weights' rounding and float32 arithmetic.

Operands of the history. Rotated query row: scaled by a power of two (compact metadata: by the groups' steps too) and
rounded to fp16. Keys and values: code scale + zero, rounded to fp16 once; the codebook's scale is the range times 256/255
rounded to fp16 (its levels are k / 256); compact ones are whole multiples of half a step, not rounded.

Bound. A weight's rounding to fp16 is off by 2^-11 of it at most, spread over its interval: o moves with a variance of
sum p_t^2 v_t^2 2^-22 / 3, of thousands of terms, and 8 deviations are not passed once in 10^15; 2 % more for rotated query
channels within float32's error of an fp16 tie. Float32: 2^-18 of the output; with V rotated also 135 additions of the
product with R_V^T, 135 2^-24 < 2^-16 of the sum's length."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    from gpu_cases import DEV, build_decode_case, pool_from_device, to_dev_bf16
    from test_gpu_tree import compare, dev, draft
import synth
from oracle import pool as P
from oracle.rotation import composite_rotation
from tree_cases import mask_words, random_mask


def history_values(pm, prm, h, lh, hist_pt):
    """K and V of the history's tokens [lh, 128] as the kernel feeds them to the products."""
    geo = pm.geo
    out = [[], []]
    for i in range(-(-lh // 64)):
        rows = np.arange(min(64, lh - 64 * i))
        kc, ka, kb, vc, va, vb = pm.read_history(int(hist_pt[i]), rows, h)
        for kind, (c, a, b) in enumerate(((kc, ka, kb), (vc, va, vb))):
            if geo.meta_format == "u8":
                out[kind].append(P.dequant_rows(c, a, b, prm, kind, geo))
                continue
            scale, zero = (np.asarray(x, np.float16).astype(np.float32) for x in (a, b))
            level = np.asarray(c).astype(np.float64)
            if geo.meta_format == "cb":
                scale = (scale * np.float32(256 / 255)).astype(np.float16)
                level = np.asarray(prm.cb_v if kind else prm.cb_k).astype(np.float64)[np.asarray(c).astype(int)] / 256
            x = level * np.repeat(scale.astype(np.float64), 64, 1) + np.repeat(zero.astype(np.float64), 64, 1)
            out[kind].append(x.astype(np.float16).astype(np.float64))
    return [np.concatenate(x) for x in out]


def reference(pm, prm, L, hist_pt, bf16_pt, q, kd, vd, mask, sm, v_mode):
    """(o, bound) of one request with one kv head."""
    n, hq, d = q.shape
    p = prm[0]
    seg, kk, vv = P.gather_request(pm, L, hist_pt, bf16_pt, heads=[0], params=prm)
    hist = np.array([s == "history" for s in seg] + [False] * n, bool)
    k, v = np.concatenate([kk[:, 0], kd[:, 0]]), np.concatenate([vv[:, 0], vd[:, 0]])
    k[hist], v[hist] = history_values(pm, p, 0, int(hist.sum()), hist_pt)
    rk, rv = (composite_rotation(np.asarray(x, np.float64)) for x in (p.u_k, p.u_v))
    if v_mode:
        v[hist] = v[hist] @ rv.T
    unit = np.ones(d)
    if pm.geo.meta_format == "u8":
        unit = np.repeat(p.tau_k.reshape(2, -1).max(1), 64).astype(np.float32)
        unit = unit / unit.max()
    o, bound = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        see = np.concatenate([np.ones(L, bool), mask[i]])
        for e in range(hq):
            qr = (q[i, e] @ rk).astype(np.float32)
            scale = 2.0 ** (10 - np.frexp(np.abs(qr).max())[1])
            qr = (qr * (np.float32(scale) * unit)).astype(np.float16).astype(np.float64) / (scale * unit)
            x = np.where(hist, k @ qr, k @ q[i, e])[see] * sm
            w = np.exp(x - x.max())
            w /= w.sum()
            o[i, e] = w @ v[see]
            dev_ = np.sqrt((w * hist[see]) ** 2 @ v[see] ** 2 * 2.0 ** -22 / 3)
            bound[i, e] = 8.2 * dev_ + 2.0 ** -18 * np.abs(o[i, e]) + 2.0 ** -21
            if v_mode:
                bound[i, e] += 2.0 ** -16 * np.linalg.norm((w * hist[see]) @ v[see])
    return o, bound


@pytest.mark.parametrize("meta,v_mode", [("f16", 0), ("f16", 1), ("u8", 1), ("cb", 0), ("cb", 1)])
@pytest.mark.parametrize("T", [20, 40])
def test_error_is_what_the_roundings_make(meta, v_mode, T):
    lens, hkv, gq = [6011], 1, 4
    case = build_decode_case(lens, hkv, gq, v_mode, seed=74, meta=meta)
    q, kd, vd = draft(74, 1, T, hkv, gq)
    mask = random_mask(np.random.default_rng(4), 1, T, "tree")
    cache, prm, hp, bp = case
    out = cache.tree_attention(0, *(to_dev_bf16(x) for x in (q, kd, vd)), torch.from_numpy(mask_words(mask)).to(DEV), dev(lens), hp,
                               bp, synth.sm_scale(), out_dtype=osc.OUT_FP32)
    assert cache.get_status() == 0
    compare(out, None, case, lens, q, kd, vd, mask, [T], v_mode, synth.sm_scale())
    o, bound = reference(pool_from_device(cache, 0), prm, lens[0], hp[0], bp[0], *(x[0].astype(np.float64) for x in (q, kd, vd)),
                         mask[0], synth.sm_scale(), v_mode)
    off = np.abs(out[0].double().cpu().numpy() - o)
    assert (off <= bound).all(), (off / bound).max()
