"""64-bit causal attention and the rounding bound of the prompt attention, shared by its GPU tests.

Bound. A logit x = F (q . k) (F = scale log2 e) is a float32 tensor-core sum of exact products, off by at most 2^-19 of
F sum |q_c k_c| (128 products, truncated sums), and its difference to the reference is rounded once (2^-23 of |x| and the
reference's size): in all less than 2^-18 F |q| |k|max. With e = ln 2 times that plus 2^-21 (the exponential and the sum), a
weight is off by e, and rounded once to bf16: half a step, 2^-8. The result is sum p v / sum p, its numerator summed by the
tensor cores with truncation (measured 2e-5 of the mean at 32K tokens: 2^-26 for every 16 tokens, four times that here): off
by (2^-8 + 2 e + n 2^-28) (1 + 2^-8) A with A = sum p |v| / sum p. A bf16 result is rounded once more. lse: e / 1, and float32's
rounding of its parts, 2^-22 of the largest.
"""
import math

import torch


def reference(q, k, v, lens, starts, scale, rows=None):
    """Per prompt and row (out, bound of out before its rounding, lse, bound of lse), float64 on the CPU: dicts by row index;
    rows: the tokens of the buffer that are wanted (None: all)."""
    q, k, v = (x.double().cpu() for x in (q, k, v))
    gq = q.shape[1] // k.shape[1]
    F = scale / math.log(2)
    found = []
    for n, at in zip(lens, starts):
        mine = [i for i in range(n) if rows is None or at + i in rows]
        if not mine:
            continue
        idx = torch.tensor(mine)
        kk, vv = (x[at:at + n].repeat_interleave(gq, 1) for x in (k, v))       # [n, hq, 128]
        x = torch.einsum("qhd,khd->hqk", q[at + idx], kk) * scale
        later = torch.arange(n) > idx[:, None]
        x = x.masked_fill(later, -math.inf)
        p = torch.softmax(x, -1)
        vm = vv.masked_fill(vv.isnan(), 0.0)
        out, A = torch.einsum("hqk,khd->qhd", p, vm), torch.einsum("hqk,khd->qhd", p, vm.abs())
        e = math.log(2) * 2.0 ** -18 * F * q[at + idx].norm(dim=-1) * kk.norm(dim=-1).max() + 2.0 ** -21
        lse = torch.logsumexp(x, -1).T
        bound = (2.0 ** -8 + 2 * e[..., None] + n * 2.0 ** -28) * (1 + 2.0 ** -8) * A
        found.append((at + idx, out, bound, lse, e + 2.0 ** -22 * (lse.abs() + F * 1.0 + 1.0)))
    return [torch.cat(t) for t in zip(*found)]


def check(out, lse, q, k, v, lens, starts, scale, rows=None):
    idx, want, bound, want_lse, bound_lse = reference(q, k, v, lens, starts, scale, rows)
    got = out[idx.to(out.device)].double().cpu()
    if out.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8
    off = (got - want).abs()
    assert (off <= bound + 1e-37).all(), ((off / bound).max().item(), got.isnan().sum().item())
    if lse is not None:
        off = (lse[idx.to(out.device)].double().cpu() - want_lse).abs()
        assert (off <= bound_lse).all(), (off / bound_lse).max().item()
