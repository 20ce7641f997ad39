"""64-bit references and rounding bounds of the row operators (rotation with several axes, norm with rotation, its
gradient), shared by the GPU tests.

Bounds. A turned value s (a cos t - b sin t) is off by at most s (|a| + |b|) 2^-20.5 before its last rounding (derived
in test_gpu_rope.py). The norm's factor r: a lane adds up to 32 squares, groups five more times, then the mean, eps
and a reciprocal square root of 2 units in the last place: relative (40 + 3) / 2 2^-24 + 2^-22 < 26 2^-24; times w and x
two more roundings: a normed value is off by less than 2^-19 of itself, a turned one by s (|a| + |b|) 2^-18.5. The result is
then rounded once: half a step.

Gradient. With H = s (|ga| + |gb|) for h (|h|'s bound, passed channels: |g|), u = h w and c = r^2 mean(u x): every term of
c has the error of h (2^-20.5), two products (2^-23) and a sum of up to 40 roundings, r^2 2^-18.9 more, so c is off by less
than r^2 mean(H |w| |x|) 2^-18; r (u - x c) adds four roundings and r's own error. Together
r (H |w| + |x| r^2 mean(H |w| |x|)) 2^-17.5 before the last rounding. A weight's sum of terms h x r, each off by 2^-18.5 of
H |x| r, passes a lane's chain of `chain` additions and about 100 more of warps and CTAs: sum(H |x| r) (2^-18.5 + (chain + 100) 2^-24).
"""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def pairs_of(rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == 0 else (2 * i, 2 * i + 1)


def angles(plan, pos):
    """float64 [N, 1, pairs] of positions [N] or [A, N], from 80-bit turns."""
    pos = np.asarray(pos, np.int64).reshape(-1, np.shape(pos)[-1])
    axes = np.zeros(len(plan.inv_freq), np.int64) if plan.axes is None else plan.axes.cpu().numpy().astype(np.int64)
    turn = np.longdouble(pos[axes].T) * (np.longdouble(plan.inv_freq) / (2 * np.longdouble(np.pi)))
    return torch.from_numpy(np.float64((turn - np.floor(turn)) * 2 * np.longdouble(np.pi)))[:, None]


def turned(y, plan, pos, layout, inverse=False):
    """(rotated rows, s (|a| + |b|) of each channel; a passed channel: its size) in 64 bits."""
    y = y.clone()
    t = angles(plan, pos) * (-1 if inverse else 1)
    a, b = pairs_of(plan.rotary_dim, layout)
    u, v, size = y[..., a].clone(), y[..., b].clone(), y.abs()
    size[..., a] = size[..., b] = abs(plan.scale) * (u.abs() + v.abs())
    y[..., a], y[..., b] = plan.scale * (u * t.cos() - v * t.sin()), plan.scale * (v * t.cos() + u * t.sin())
    return y, size


def rounded(want, off, dtype):
    """Bound after the one rounding to dtype of a value within `off` of want."""
    eps = torch.finfo(dtype).eps / 2
    return off * (1 + eps) + want.abs() * eps + torch.finfo(dtype).tiny * eps


def weight64(w, dim):
    return torch.ones(dim, dtype=torch.float64) if w is None else w.double().cpu()


def normed(x, w, eps):
    x = x.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r * weight64(w, x.shape[-1]), r


def norm_rope(x, w, eps, plan, pos, layout):
    y, size = turned(normed(x, w, eps)[0], plan, pos, layout)
    return y, rounded(y, size * 2.0 ** -18.5, x.dtype)


def norm_rope_grad(x, g, w, eps, plan, pos, layout, chain):
    """((dx, bound), (dw, bound))"""
    (_, r), x64, w64 = normed(x, w, eps), x.double().cpu(), weight64(w, x.shape[-1])
    h, H = turned(g.double().cpu(), plan, pos, layout, inverse=True)
    live = torch.as_tensor(np.asarray(pos).reshape(-1, len(x)).min(0) >= 0)[:, None, None]
    h, H = h * live, H * live
    c = r ** 2 * (h * w64 * x64).mean(-1, keepdim=True)
    C = r ** 2 * (H * w64.abs() * x64.abs()).mean(-1, keepdim=True)
    dx = r * (h * w64 - x64 * c)
    off = r * (H * w64.abs() + x64.abs() * C) * 2.0 ** -17.5
    dw, size = (h * x64 * r).sum((0, 1)), (H * x64.abs() * r).sum((0, 1))
    return (dx, rounded(dx, off, x.dtype)), (dw, size * (2.0 ** -18.5 + (chain + 100) * 2.0 ** -24) + 1e-38)


def near(got, want, bound, what=""):
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), (what, (off / bound).max().item())
