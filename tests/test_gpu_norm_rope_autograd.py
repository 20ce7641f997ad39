"""norm_rope and norm_rope_backward inside a torch.autograd.Function, as a training program wraps them: gradients against the
64-bit formulas (bounds: layer_cases.py), on the default stream and on another."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import layer_cases as L  # noqa: E402

if torch.cuda.is_available():
    import bit_kv_cache_decode_gb300 as osc
    DEV = torch.device("cuda:0")


class NormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, plan, positions):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        ctx.plan = plan
        return osc.norm_rope(plan, q, k, positions, q_weight, k_weight)

    @staticmethod
    def backward(ctx, grad_q, grad_k):
        q, k, qw, kw, pos = ctx.saved_tensors
        dq, dk, dqw, dkw = osc.norm_rope_backward(ctx.plan, q, k, pos, grad_q.contiguous(), grad_k.contiguous(), qw, kw)
        return dq, dk, dqw.to(qw.dtype), dkw.to(kw.dtype), None, None


@pytest.mark.parametrize("other_stream", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_through_autograd(dtype, other_stream):
    g = torch.Generator(device=DEV).manual_seed(4)
    N, hq, hkv, dtype = 203, 6, 2, getattr(torch, dtype)
    x = torch.randn(N, (hq + hkv) * 128, generator=g, device=DEV).to(dtype).requires_grad_()
    w = (1 + 0.3 * torch.randn(2, 128, generator=g, device=DEV)).to(dtype).requires_grad_()
    c = torch.randn(N, hq + hkv, 128, generator=g, device=DEV).to(dtype)
    pos, plan = torch.randint(0, 10 ** 5, (N,), generator=g, device=DEV, dtype=torch.int32), osc.RopePlan(128, base=1e6)
    stream = torch.cuda.Stream() if other_stream else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q, k = x.unflatten(1, (-1, 128)).split([hq, hkv], 1)             # views of one projection
        yq, yk = NormRope.apply(q, k, w[0], w[1], plan, pos)
        ((yq.float() * c[:, :hq].float()).sum() + (yk.float() * c[:, hq:].float()).sum()).backward()
    stream.synchronize()
    grad = x.grad.view(N, hq + hkv, 128)
    for i, (rows, y) in enumerate(((slice(0, hq), yq), (slice(hq, hq + hkv), yk))):
        xx = x.detach().view(N, -1, 128)[:, rows]
        L.near(y.detach(), *L.norm_rope(xx, w[i].detach(), 1e-6, plan, pos.cpu(), 0), "forward")
        # a lane's chain: no longer than all rows of its CTA
        (dx, bx), (dw, bw) = L.norm_rope_grad(xx, c[:, rows], w[i].detach(), 1e-6, plan, pos.cpu(), 0, N * hq)
        L.near(grad[:, rows], dx, bx, "dx")
        L.near(w.grad[i], dw, L.rounded(dw, bw, dtype), "dw")
