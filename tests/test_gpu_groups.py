"""GPU tests of the router that chooses groups of experts first, against the
float64 reference: the choice exactly, weights and gradient as route()'s."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref  # noqa: E402
import more_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
INF = math.inf


def check(x, k, groups, top, best, score="softmax", bias=None, renormalise=True, scale=1.0, grad=True):
    t, e = x.shape
    print(f"[gpu-case] route {t}x{e} top {k} of {top}/{groups} groups best={best} {score} {x.dtype} "
          f"bias={bias is not None} renormalise={renormalise}", flush=True)
    how = dict(score=score, renormalise=renormalise, scale=scale)
    ids, w = mg.route(x.cuda(), k, bias=None if bias is None else bias.cuda(), num_groups=groups, top_groups=top,
                      group_best=best, **how)
    want = ref.route_grouped(x, k, groups, top, best, score, bias)
    assert torch.equal(ids.cpu().long(), want), (ids.cpu().long() != want).any(1).nonzero()[:4].tolist()
    xd = x.double().clamp(max=torch.finfo(torch.float32).max)
    if score == "softmax":
        m = torch.where(xd > -INF, xd, -INF).amax(1, keepdim=True)
        ex = torch.where(xd == -INF, 0.0, torch.exp(xd - torch.where(m == -INF, 0.0, m)))
        p = ex / ex.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.exp(-torch.logaddexp(torch.zeros_like(xd), -xd))
    ww = layer_ref.weights_of(xd, want, p, score, renormalise, scale)
    # exponentials of arguments up to |l - max| off by their rounding, sums of up to 1024, a division
    off = 64 * ref.F32 * (1.0 + xd.abs().where(xd.abs() < 1e30, 0.0).amax()) * ww.abs() + 1e-37
    assert ((w.cpu().double() - ww).abs() <= off).all()
    if grad:
        gen = torch.Generator().manual_seed(5)
        g = torch.randn(t, k, generator=gen)
        d = mg.route_backward(x.cuda(), ids, g.cuda(), **how).cpu().double()
        dd = layer_ref.route_backward(x, want, g, score, renormalise, scale)
        eps = ref.BF16 if x.dtype == torch.bfloat16 else ref.F32
        most = (g.abs().sum(1, keepdim=True) * abs(scale)).double()
        assert ((d - dd).abs() <= eps * dd.abs() + 256 * ref.F32 * most + 1e-37).all()
    return ids, w


def check_up_to_64_bits(x, k, groups, top, best, score, bias):
    """As check() of the ids, where scores may be nearer than 64 bits tell.  With v = 2^-53: a score is an
    exponential (2 v of it), a sum and a quotient (v each; the softmax's sum of at most 1024 terms, by
    partial sums of at most 16 + 6, 24 v), so p is off by at most 30 v in either order of the operations, p +
    bias by 2 v more (|p + bias| < 2), and a sum of two keys by 2 * 32 v + 2 v: numbers nearer than twice that,
    132 v < 2^-45, can stand in either order.  Logits are exact.  Such a row's choice has to be one that
    some order of such numbers gives."""
    t, e = x.shape
    size, near = e // groups, 2.0 ** -45
    print(f"[gpu-case] route {t}x{e} top {k} of {top}/{groups} groups best={best} {score} bias={bias is not None}", flush=True)
    ids, _ = mg.route(x.cuda(), k, score=score, bias=None if bias is None else bias.cuda(), num_groups=groups,
                      top_groups=top, group_best=best)
    ids = ids.cpu().long()
    want = ref.route_grouped(x, k, groups, top, best, score, bias)
    for i in (ids != want).any(1).nonzero().flatten().tolist():
        l = x[i].double()
        p = torch.where(l > -INF, torch.softmax(l, 0) if score == "softmax" else torch.sigmoid(l), 0.0)
        key = torch.where(l > -INF, l if bias is None else p + bias.double(), -INF)
        base = key if bias is not None or best == 1 else torch.where(l > -INF, p, -INF)
        two = base.reshape(groups, size).topk(best, 1).values
        g = torch.where(two[:, -1] > -INF, two.sum(1), two[:, 0])
        edge = g.sort(descending=True).values[top - 1]
        sharp = bias is None and best == 1
        assert not sharp, i
        sure = [q for q in range(groups) if g[q] > edge + near]
        maybe = [q for q in range(groups) if abs(g[q] - edge) <= near]
        fits = False
        for some in itertools.combinations(maybe, top - len(sure)):
            open_ = torch.zeros(groups, dtype=torch.bool)
            open_[list(sure) + list(some)] = True
            kk = torch.where(open_.repeat_interleave(size), key, -INF)
            if bias is None:
                order = sorted((j for j in range(e) if kk[j] > -INF), key=lambda j: (-kk[j].item(), j))[:k]
                fits |= ids[i].tolist() == order + [-1] * (k - len(order))
            else:
                got = [j for j in ids[i].tolist() if j >= 0]
                v, left = kk[got], kk.clone()
                left[got] = -INF
                fits |= len(set(got)) == len(got) == min(k, int((kk > -INF).sum())) and bool(
                    (v > -INF).all() and (v[1:] <= v[:-1] + near).all() and (len(got) == 0 or left.max() <= v[-1] + near))
        assert fits, (i, ids[i].tolist(), want[i].tolist())


def logits(t, e, seed, dtype=torch.float32, spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(t, e, generator=gen) * spread).to(dtype), gen


SHAPES = [(1, 4, 1, 2, 1), (5, 64, 6, 8, 3), (33, 60, 4, 5, 2), (100, 256, 8, 8, 4), (17, 160, 6, 8, 3), (64, 128, 2, 64, 5),
          (40, 96, 12, 3, 1), (9, 1024, 32, 16, 5), (21, 1000, 3, 8, 7), (30, 64, 7, 64, 9), (12, 320, 5, 64, 64),
          (3, 512, 9, 1, 1), (1000, 36, 3, 4, 3)]


@pytest.mark.parametrize("t,e,k,groups,top", SHAPES)
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_choice(t, e, k, groups, top, best, score, with_bias, dtype):
    x, gen = logits(t, e, t + e + best, dtype)
    bias = torch.randn(e, generator=gen) * 0.2 if with_bias else None
    check(x, k, groups, top, best, score, bias, renormalise=(t + k) % 2 == 0, scale=1.0 if best == 1 else 2.5)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties(best, score, with_bias):
    """Few different logits: groups and experts of equal scores, the lowest index first."""
    gen = torch.Generator().manual_seed(best)
    x = torch.randint(-2, 3, (600, 48), generator=gen).float() * 0.5
    bias = torch.randint(-1, 2, (48,), generator=gen).float() * 0.25 if with_bias else None
    check(x, 5, 6, 2, best, score, bias)
    check(torch.zeros(7, 48), 5, 6, 2, best, score, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_next_to_each_other(score):
    """Groups whose scores differ in the last bits of 64 alone, or in bits that fp32 sums lose."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(400, 1, generator=gen).expand(400, 64).contiguous()
    x = x * (1.0 + torch.randint(-3, 4, (400, 64), generator=gen) * 2.0 ** -22)
    check(x, 4, 8, 3, 2, score)
    bias = 1.0 + torch.randint(-4, 5, (64,), generator=gen) * 2.0 ** -22
    check(x, 4, 8, 3, 2, score, bias)
    check(x, 4, 8, 3, 1, score, bias)
    # pairs that swap their members' bits between them: sums equal in exact numbers
    check(torch.cat([x[:, :32], x[:, :32].flip(1)], 1), 4, 8, 3, 2, score)


@pytest.mark.parametrize("t,e,groups,top", [(300, 60, 5, 2), (200, 1000, 8, 3), (200, 640, 5, 2), (2100, 256, 8, 4), (300, 256, 8, 4),
                                            (2100, 160, 8, 3), (2100, 120, 10, 4), (100, 1024, 16, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_scores_next_to_each_other_of_all_shapes(t, e, groups, top, score, with_bias):
    """The same for groups of whole lanes, of parts of them and of more than 32 experts: all of a token's
    experts within a few steps of fp32, empty groups among them."""
    gen = torch.Generator().manual_seed(e + t)
    x = torch.randn(t, 1, generator=gen).expand(t, e).contiguous()
    x = x * (1.0 + torch.randint(-3, 4, (t, e), generator=gen) * 2.0 ** -22)
    x[1::4] = torch.where(torch.rand(x[1::4].shape, generator=gen) < 0.9, -INF, x[1::4])
    x[2::4, :e // groups] = -INF
    x[3::4] += torch.rand(x[3::4].shape, generator=gen) * 1e-5
    bias = 0.25 + torch.randint(-4, 5, (e,), generator=gen) * 2.0 ** -24 if with_bias else None
    for best in (1, 2):
        check_up_to_64_bits(x, 6, groups, top, best, score, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(score, best, with_bias):
    x, gen = logits(300, 64, 9)
    x[torch.rand(300, 64, generator=gen) < 0.6] = -INF
    x[:20, 8:] = -INF                                   # one group has all that is left
    x[20:40] = -INF                                     # nothing is left
    x[40:60, ::2] = -INF
    x[60:70, 3] = INF
    x[70:80, 16:24] = -1e30
    x[80:90, :48] = torch.finfo(torch.float32).min      # the lowest number is one that can be chosen
    bias = torch.randn(64, generator=gen) * 0.1 if with_bias else None
    if with_bias:
        bias[5], bias[9], bias[17] = math.nan, -INF, 30.0
    check(x, 6, 8, 3, best, score, bias)
    check(x, 6, 8, 3, best, score, bias, renormalise=score == "sigmoid", grad=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_not_numbers(score, best):
    """An expert whose logit is NaN is never chosen and leaves the groups' scores alone."""
    x, gen = logits(100, 40, 4)
    x[::3, 7] = math.nan
    x[1, :] = math.nan
    ids, _ = mg.route(x.cuda(), 3, score=score, num_groups=5, top_groups=2, group_best=best)
    assert torch.equal(ids.cpu().long(), ref.route_grouped(x, 3, 5, 2, best, score))
    bias = torch.randn(40, generator=gen)
    ids, _ = mg.route(x.cuda(), 3, score=score, bias=bias.cuda(), num_groups=5, top_groups=2, group_best=best)
    assert torch.equal(ids.cpu().long(), ref.route_grouped(x, 3, 5, 2, best, score, bias))


def test_all_groups_are_no_choice():
    x, gen = logits(200, 64, 1)
    bias = (torch.randn(64, generator=gen) * 0.1).cuda()
    a = mg.route(x.cuda(), 6, bias=bias)
    for groups in (2, 8, 64):
        b = mg.route(x.cuda(), 6, bias=bias, num_groups=groups, top_groups=groups, group_best=2)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_large_batch():
    x, gen = logits(5003, 256, 2, torch.bfloat16)
    check(x, 8, 8, 4, 2, "sigmoid", torch.randn(256, generator=gen) * 0.1)


@pytest.mark.parametrize("t", [2048, 2049])
@pytest.mark.parametrize("e,groups,top", [(72, 8, 3), (128, 8, 4), (160, 8, 3), (256, 16, 5), (256, 2, 1)])
@pytest.mark.parametrize("score,best,with_bias", [("softmax", 1, False), ("softmax", 2, True), ("sigmoid", 2, False)])
def test_few_tokens_and_many(t, e, groups, top, score, best, with_bias):
    """Up to 2048 tokens of up to 256 experts go a wave a token, more by four to a wave."""
    x, gen = logits(t, e, t + e, torch.bfloat16)
    x[::5, ::3] = -INF
    check(x, 5, groups, top, best, score, torch.randn(e, generator=gen) * 0.1 if with_bias else None)


@pytest.mark.parametrize("t", [2048, 2049])
@pytest.mark.parametrize("e", [65, 96, 128, 200, 256])
@pytest.mark.parametrize("score,with_bias", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("renormalise", [False, True])
def test_without_groups_few_tokens_and_many(t, e, score, with_bias, renormalise):
    x, gen = logits(t, e, t + e)
    bias = torch.randn(e, generator=gen) * 0.1 if with_bias else None
    print(f"[gpu-case] route {t}x{e} {score} bias={with_bias} renormalise={renormalise}", flush=True)
    ids, w = mg.route(x.cuda(), 7, score=score, bias=None if bias is None else bias.cuda(), renormalise=renormalise)
    want, ww, _ = layer_ref.route(x, 7, score, bias, renormalise)
    assert torch.equal(ids.cpu().long(), want)
    assert ((w.cpu().double() - ww).abs() <= 64 * ref.F32 * (1.0 + x.abs().amax()) * ww.abs()).all()
    g = torch.randn(t, 7, generator=gen)
    d = mg.route_backward(x.cuda(), ids, g.cuda(), score=score, renormalise=renormalise).cpu().double()
    dd = layer_ref.route_backward(x, want, g, score, renormalise)
    assert ((d - dd).abs() <= ref.F32 * dd.abs() + 256 * ref.F32 * g.abs().sum(1, keepdim=True).double()).all()


@pytest.mark.parametrize("t", [37, 2051])
@pytest.mark.parametrize("e,groups,top", [(256, 8, 1), (256, 8, 4), (256, 16, 8), (128, 8, 2), (1024, 16, 8), (512, 8, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_keys_of_few_groups(t, e, groups, top, with_bias):
    """Open groups that are at most half of the lanes, whose keys are dealt out: equal and masked
    experts, more choices than experts that are left, the last expert of a lane."""
    gen = torch.Generator().manual_seed(t + e + top)
    x = torch.randint(-3, 4, (t, e), generator=gen).float() * 0.5
    x[::4] = torch.randn((t + 3) // 4, e, generator=gen)
    x[1::4, ::2] = -INF
    x[2::4] = torch.where(torch.rand(x[2::4].shape, generator=gen) < 0.95, -INF, x[2::4])
    x[3::8] = 0.0
    x[7::8, ::3] = -0.0                                 # (0 and -0 are one number)
    bias = torch.randint(-1, 2, (e,), generator=gen).float() * 0.25 if with_bias else None
    for k in (1, 8, 16, 31):
        if k <= top * (e // groups):
            check(x, k, groups, top, 2, "sigmoid", bias, grad=False)


@pytest.mark.parametrize("t", [5, 2100])
@pytest.mark.parametrize("e", [40, 70, 128, 256, 600])
@pytest.mark.parametrize("k", [4, 20])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_of_an_expert_chosen_twice(t, e, k, renormalise):
    """Ids that a caller has changed: the gradients of equal ones are added, those out of range have none."""
    x, gen = logits(t, e, t + e + k)
    ids = torch.randint(-1, e + 1, (t, k), generator=gen, dtype=torch.int32)
    ids[::3, 1] = ids[::3, 0]
    ids[1::3] = torch.stack([torch.randperm(e, generator=gen)[:k] for _ in range(ids[1::3].shape[0])]).int()
    g = torch.randn(t, k, generator=gen)
    for score in ("softmax", "sigmoid"):
        d = mg.route_backward(x.cuda(), ids.cuda(), g.cuda(), score=score, renormalise=renormalise).cpu().double()
        dd = layer_ref.route_backward(x, ids, g, score, renormalise)
        assert ((d - dd).abs() <= ref.F32 * dd.abs() + 256 * ref.F32 * g.abs().sum(1, keepdim=True).double()).all()


def test_no_tokens_and_graph():
    ids, w = mg.route(torch.empty(0, 64, device="cuda"), 4, num_groups=8, top_groups=2)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    x, gen = logits(777, 256, 2)
    x, bias = x.cuda(), (torch.randn(256, generator=gen) * 0.1).cuda()
    how = dict(bias=bias, score="sigmoid", num_groups=8, top_groups=4, group_best=2)
    want = mg.route(x, 8, **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mg.route(x, 8, stream=side, **how)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mg.route(x, 8, **how)
    for _ in range(3):
        got[0].zero_(), got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        torch.randn(100000, device="cuda").sum().item()
