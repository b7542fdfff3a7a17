"""GPU tests of the router on both sides of the number of tokens up to which a
wave has a token (1024 of 65 to 128 experts, 2048 of up to 256)."""
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref  # noqa: E402
import more_ref as ref  # noqa: E402
from test_gpu_groups import check  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("t", [1024, 1025])
@pytest.mark.parametrize("e", [65, 96, 120, 128])
@pytest.mark.parametrize("score,with_bias", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_of_up_to_128_experts(t, e, score, with_bias, dtype):
    gen = torch.Generator().manual_seed(t + e)
    x = (torch.randn(t, e, generator=gen) * 1.5).to(dtype)
    x[::7, ::3] = -INF
    x[3] = 0.0
    bias = torch.randn(e, generator=gen) * 0.1 if with_bias else None
    print(f"[gpu-case] route {t}x{e} {score} bias={with_bias} {dtype}", flush=True)
    for renormalise in (False, True):
        how = dict(score=score, renormalise=renormalise)
        ids, w = mg.route(x.cuda(), 7, bias=None if bias is None else bias.cuda(), **how)
        want, ww, _ = layer_ref.route(x, 7, score, bias, renormalise)
        assert torch.equal(ids.cpu().long(), want)
        assert ((w.cpu().double() - ww).abs() <= 64 * ref.F32 * 10.0 * ww.abs()).all()      # |l| < 9
        g = torch.randn(t, 7, generator=gen)
        d = mg.route_backward(x.cuda(), ids, g.cuda(), **how).cpu().double()
        dd = layer_ref.route_backward(x, want, g, score, renormalise)
        eps = ref.BF16 if dtype == torch.bfloat16 else ref.F32
        assert ((d - dd).abs() <= eps * dd.abs() + 256 * ref.F32 * g.abs().sum(1, keepdim=True).double()).all()


@pytest.mark.parametrize("t", [1024, 1025])
@pytest.mark.parametrize("e,groups,top", [(72, 8, 3), (96, 6, 2), (120, 40, 11), (128, 8, 4), (128, 2, 1)])
@pytest.mark.parametrize("score,best,with_bias", [("softmax", 1, False), ("softmax", 2, True), ("sigmoid", 2, False)])
def test_groups_of_up_to_128_experts(t, e, groups, top, score, best, with_bias):
    gen = torch.Generator().manual_seed(t + e)
    x = (torch.randn(t, e, generator=gen) * 1.5).to(torch.bfloat16)
    x[::5, ::3] = -INF
    check(x, 5, groups, top, best, score, torch.randn(e, generator=gen) * 0.1 if with_bias else None)
