"""GPU tests of the router: every output against the float64 reference."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
U = ref.F32


def make(t, e, dtype, seed, masked=True, spread=2.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, e, generator=gen) * spread
    if masked:
        x[torch.rand(t, e, generator=gen) < 0.1] = -math.inf
        x[torch.rand(t, generator=gen) < 0.1] = -math.inf
    return x.to(dtype), torch.randn(e, generator=gen) * 0.2, gen


def check(x, k, score, bias, renorm, scale, gen):
    """Forward and backward of one call against the reference."""
    t, e = x.shape
    print(f"[gpu-case] route {t}x{e} k={k} {x.dtype} {score} bias={bias is not None} renorm={renorm}", flush=True)
    how = dict(score=score, renormalise=renorm, scale=scale)
    ids, w = mg.route(x.cuda(), k, bias=None if bias is None else bias.cuda(), **how)
    rid, rw, p = ref.route(x, k, score, bias, renorm, scale)
    assert torch.equal(ids.cpu().long(), rid)
    # exp of a rounded difference, a sum of e terms, a few roundings
    size = torch.where(x.float().abs() < 1e30, x.float().abs(), 0.0).double().amax(1, keepdim=True)
    rel = (e + 32 + 4 * size) * U
    assert torch.equal(torch.isnan(w.cpu()), torch.isnan(rw))
    ok = ~torch.isnan(rw)
    assert ((w.cpu().double() - rw).abs() <= rel * rw.abs() + 1e-37)[ok].all()
    g = torch.randn(t, k, generator=gen)
    d = mg.route_backward(x.cuda(), ids, g.cuda(), **how).cpu()
    rd = ref.route_backward(x, rid, g, score, renorm, scale)
    assert d.dtype == x.dtype
    # a difference of terms up to scale |g| each, times the weight's or score's error
    big = abs(scale) * g.double().abs().amax(1, keepdim=True)
    if renorm or score == "sigmoid":
        lead = torch.zeros(t, e, dtype=torch.float64).scatter_add_(1, rid.clamp(min=0), rw.abs())
        lead = lead * (k if renorm else 1) * g.double().abs().amax(1, keepdim=True)
    else:
        lead = p * big * k
    eps = ref.BF16 if d.dtype == torch.bfloat16 else U
    good = ~torch.isnan(rd)
    assert torch.equal(torch.isnan(d), ~good)
    assert ((d.double() - rd).abs() <= (eps * rd.abs() + 4 * rel * lead + 1e-37))[good].all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("t,e,k,dtype", [
    (1, 64, 6, torch.float32), (5, 8, 8, torch.bfloat16), (3, 1, 1, torch.float32), (37, 7, 2, torch.bfloat16),
    (130, 60, 4, torch.float32), (65, 100, 5, torch.bfloat16), (1001, 128, 8, torch.bfloat16),
    (33, 129, 3, torch.float32), (250, 256, 8, torch.bfloat16), (17, 384, 32, torch.float32),
    (40, 1000, 10, torch.bfloat16), (19, 1024, 16, torch.float32), (70, 257, 2, torch.bfloat16),
])
def test_route(t, e, k, dtype, score, renorm, biased):
    if biased:
        spread = 2.0
    x, bias, gen = make(t, e, dtype, seed=t * 7 + e, masked=t > 1, spread=2.0)
    check(x, k, score, bias if biased else None, renorm, 1.0 if renorm else 2.5, gen)


def test_route_many_tokens():
    x, bias, gen = make(16381, 256, torch.bfloat16, seed=5)
    check(x, 8, "sigmoid", bias, True, 1.0, gen)


def test_route_ties_go_to_the_lowest_index():
    x = torch.zeros(4, 200)
    x[1, 150:] = 1.0
    x[2, ::3] = -1.0
    x[3] = torch.arange(200) % 2 * 1.0
    for bias in (None, torch.zeros(200)):
        for score in ("softmax", "sigmoid"):
            ids, _ = mg.route(x.cuda(), 6, score=score, bias=None if bias is None else bias.cuda())
            assert ids[0].tolist() == [0, 1, 2, 3, 4, 5]
            assert ids[1].tolist() == [150, 151, 152, 153, 154, 155]
            assert ids[2].tolist() == [1, 2, 4, 5, 7, 8]
            assert ids[3].tolist() == [1, 3, 5, 7, 9, 11]


def test_route_coarse_logits_with_bias():
    """Whole-number logits and biases on a grid: many exact ties of score + bias."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randint(-3, 4, (500, 256), generator=gen).to(torch.bfloat16)
    bias = torch.zeros(256)
    check(x, 8, "sigmoid", bias, True, 1.0, gen)
    check(x, 8, "softmax", bias, False, 1.0, gen)


def test_route_near_ties_are_decided_in_64_bits():
    """Keys that differ by far less than fp32 resolves."""
    x = torch.zeros(64, 64)
    x[:] = 3.0 + torch.arange(64) * 2.0 ** -21            # sigmoid(3) changes by 2e-8 a step
    perm = torch.stack([torch.randperm(64, generator=torch.Generator().manual_seed(i)) for i in range(64)])
    x = x.gather(1, perm)
    for score in ("sigmoid", "softmax"):
        ids, _ = mg.route(x.cuda(), 10, score=score, bias=torch.full((64,), 0.25).cuda())
        rid, _, _ = ref.route(x, 10, score, torch.full((64,), 0.25))
        assert torch.equal(ids.cpu().long(), rid)
        assert torch.equal(x.gather(1, rid), x.sort(1, descending=True).values[:, :10])


def test_route_special_values():
    inf, nan = math.inf, math.nan
    x = torch.tensor([[1.0, 2.0, 3.0, 0.5], [-inf] * 4, [nan, 1.0, 2.0, 0.0], [nan] * 4, [inf, 1.0, inf, 0.0],
                      [-inf, -inf, -200.0, -201.0], [3e38, -3e38, 0.0, 1.0], [-inf, nan, 5.0, -inf]])
    gen = torch.Generator().manual_seed(1)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check(x, 3, score, None, renorm, 1.0, gen)
            check(x, 3, score, torch.tensor([0.1, 0.0, -0.1, 0.05]), renorm, 1.0, gen)
    ids, w = mg.route(x.cuda(), 3, score="sigmoid")
    assert ids[1].tolist() == [-1, -1, -1] and w[1].tolist() == [0, 0, 0]
    assert ids[2].tolist() == [2, 1, 3] and ids[3].tolist() == [-1] * 3
    assert ids[5].tolist() == [2, 3, -1]
    assert abs(w[5, 0].item() - 1 / (1 + math.exp(-1))) < 1e-6     # both scores underflow in fp32
    # a bias that rules experts out
    ids, _ = mg.route(x[:1].cuda(), 3, bias=torch.tensor([0.0, -inf, nan, 0.0]).cuda())
    assert ids[0].tolist() == [0, 3, -1]


def test_route_backward_takes_foreign_ids():
    """Ids out of range have no gradient and are not followed; one that appears twice counts twice."""
    x, _, gen = make(6, 20, torch.float32, 9, masked=False)
    ids = torch.tensor([[0, 5], [-1, 3], [20, 4], [2 ** 31 - 1, -2 ** 31], [7, 7], [-1, -1]], dtype=torch.int32)
    g = torch.randn(6, 2, generator=gen)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = mg.route_backward(x.cuda(), ids.cuda(), g.cuda(), score=score, renormalise=renorm).cpu().double()
            r = ref.route_backward(x, ids, g, score, renorm)
            assert torch.allclose(d, r, rtol=1e-5, atol=1e-6)


def test_route_gradient_against_differences():
    """The GPU's gradient against differences of the GPU's own weights (fp32:
    a step of 2^-6 against an error of a few 2^-24)."""
    x, _, gen = make(8, 16, torch.float32, 4, masked=False, spread=1.0)
    g = torch.randn(8, 3, generator=gen).cuda()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            how = dict(score=score, renormalise=renorm)
            x3 = x.clone()
            x3[:, :3] += 8.0                               # the choice stays where it is
            ids, _ = mg.route(x3.cuda(), 3, **how)
            d = mg.route_backward(x3.cuda(), ids, g, **how)
            h = 2.0 ** -6
            for e in (0, 1, 2, 9):
                f = []
                for s in (h, -h):
                    y = x3.clone()
                    y[:, e] += s
                    i2, w2 = mg.route(y.cuda(), 3, **how)
                    order = (i2[:, None, :] == ids[:, :, None]).float()
                    f.append(((order @ w2[:, :, None])[:, :, 0] * g).sum(1))
                assert torch.allclose((f[0] - f[1]) / (2 * h), d[:, e], atol=2e-4)


def test_route_empty():
    ids, w = mg.route(torch.empty(0, 8, device="cuda"), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    assert mg.route_backward(torch.empty(0, 8, device="cuda"), ids, w).shape == (0, 8)
