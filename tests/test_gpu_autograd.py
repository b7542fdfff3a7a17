"""The layer operators beside autograd: no history of their own, and as what a
torch.autograd.Function calls."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


class Gated(torch.autograd.Function):
    """SwiGLU of a product, as a user wraps it."""
    @staticmethod
    def forward(ctx, x, w, b):
        y, c = mg.linear(x, w, bias=b, act="swiglu", save_c=True)
        ctx.save_for_backward(x, w, c)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, c = ctx.saved_tensors
        return mg.linear_backward(dy.contiguous(), x, w, c=c, act="swiglu")


def test_results_have_no_history():
    x = torch.randn(12, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    w = torch.randn(64, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    print("[gpu-case] operands that require gradients", flush=True)
    y = mg.linear(x, w, dtype="f32")
    ids, weights = mg.route(y.requires_grad_(), 2)
    plan = mg.sort_tokens(ids, 64, weights=weights.requires_grad_(), m_aligned=1)
    a = mg.dispatch(x, plan)
    for t in (ids, plan.prob, a, mg.combine(a, plan, weights=weights, residual=x)):
        assert not t.requires_grad and t.grad_fn is None
    assert x.grad is None and w.grad is None


def test_inside_a_function():
    """Gradients through torch's graph: each is off by at most four BF16 roundings of numbers that add up over a sum."""
    m, n, k = 150, 192, 136
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(m, k, generator=gen).to(torch.bfloat16)
    w = (torch.randn(n, k, generator=gen) / math.sqrt(k)).to(torch.bfloat16)
    b = torch.randn(n, generator=gen) * 0.1
    dy = torch.randn(m, n // 2, generator=gen).to(torch.bfloat16)
    print(f"[gpu-case] linear in an autograd function m={m} n={n} k={k}", flush=True)
    mine = [t.cuda().requires_grad_() for t in (x, w, b)]
    y = Gated.apply(*mine)
    y.backward(dy.cuda())
    them = [t.double().requires_grad_() for t in (x, w, b)]
    r = ref.act(them[0] @ them[1].t() + them[2], "swiglu")
    r.backward(dy.double())
    for g, t in zip([y, *(t.grad for t in mine)], [r.detach(), *(t.grad for t in them)]):
        assert (g.detach().cpu().double() - t).norm() <= 4 * ref.BF16 * t.norm()
