"""GPU tests of the grouped router where a lane owns up to four groups (16 lanes
a token and more than 16 groups, of 2 to 6 experts): the groups' scores decided
in 64 bits in every place of a lane, and the plain choice there."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import more_ref as ref  # noqa: E402

INF = math.inf
# numbers nearer than this can stand in either order in 64 bits: with v = 2^-53 a score is an exponential (2 v of
# it), a sum and a quotient (v each; the softmax's sum, 24 v), p + bias 2 v more, a sum of two keys 2 * 32 v + 2 v;
# twice that is 132 v < 2^-45
NEAR = 2.0 ** -45


def scores(l, groups, best, score, bias):
    """Keys of a token's experts and its groups' scores, float64."""
    l = l.double()
    some = l > -INF
    p = torch.where(some, torch.softmax(l, 0) if score == "softmax" else torch.sigmoid(l), 0.0)
    key = torch.where(some, l if bias is None else p + bias.double(), -INF)
    base = key if bias is not None or best == 1 else torch.where(some, p, -INF)
    two = base.reshape(groups, -1).topk(best, 1).values
    return key, torch.where(two[:, -1] > -INF, two.sum(1), two[:, 0])


def fits(ids, key, g, top, near_keys):
    """Whether `ids` is a choice that some order of the numbers nearer than NEAR gives: the groups that are in
    for sure, those of the others that the choice shows, and as many more as are wanted that change nothing."""
    groups, k = len(g), len(ids)
    size = len(key) // groups
    edge = g.sort(descending=True).values[top - 1]
    near = lambda v: bool(v == edge) or abs(float(v - edge)) <= NEAR
    sure = {q for q in range(groups) if g[q] > edge and not near(g[q])}
    maybe = {q for q in range(groups) if near(g[q])}
    got = [i for i in ids if i >= 0]
    seen = {i // size for i in got}
    if not seen <= sure | maybe or len(set(got)) != len(got):
        return False

    def follows(opened):
        """ids are the best of the opened groups' experts."""
        kk = torch.full_like(key, -INF)
        for q in opened:
            kk[q * size:(q + 1) * size] = key[q * size:(q + 1) * size]
        n = min(k, int((kk > -INF).sum()))
        if len(got) != n or ids[n:] != [-1] * (k - n):
            return False
        if not near_keys:
            return got == sorted((i for i in range(len(kk)) if kk[i] > -INF), key=lambda i: (-kk[i].item(), i))[:n]
        v, left = kk[got], kk.clone()
        left[got] = -INF
        return bool((v > -INF).all() and (v[1:] <= v[:-1] + NEAR).all() and (n == 0 or left.max() <= v[-1] + NEAR))
    opened = sure | seen
    spare = sum(follows(opened | {q}) for q in maybe - opened)
    return len(opened) <= top <= len(opened) + spare and follows(opened)


def check(x, k, groups, top, best, score, bias, exact=False):
    t, e = x.shape
    print(f"[gpu-case] route {t}x{e} top {k} of {top}/{groups} groups best={best} {score} bias={bias is not None}", flush=True)
    ids, w = mg.route(x.cuda(), k, score=score, bias=None if bias is None else bias.cuda(), num_groups=groups, top_groups=top,
                      group_best=best)
    ids = ids.cpu().long()
    want = ref.route_grouped(x, k, groups, top, best, score, bias)
    other = (ids != want).any(1).nonzero().flatten().tolist()
    assert not other or not (exact or (bias is None and best == 1)), other[:4]
    for i in other:
        key, g = scores(x[i], groups, best, score, bias)
        assert fits(ids[i].tolist(), key, g, top, bias is not None), (i, ids[i].tolist(), want[i].tolist())
    assert ((ids >= 0) == (w.cpu() > 0)).all()


def test_fits_takes_what_the_reference_chooses_and_nothing_else():
    """The test's own judgement: a group or an expert exchanged for a clearly worse one is refused."""
    gen = torch.Generator().manual_seed(1)
    for best in (1, 2):
        for score, with_bias in (("softmax", False), ("sigmoid", True)):
            x = torch.randn(40, 64, generator=gen)
            bias = torch.randn(64, generator=gen) * 0.1 if with_bias else None
            want = ref.route_grouped(x, 6, 32, 9, best, score, bias)
            for i in range(40):
                key, g = scores(x[i], 32, best, score, bias)
                ids = want[i].tolist()
                assert fits(ids, key, g, 9, with_bias)
                closed = int(g.argmin())
                assert not fits([2 * closed] + ids[1:], key, g, 9, with_bias)
                assert not fits([ids[1], ids[0]] + ids[2:], key, g, 9, with_bias)
                assert not fits(ids[:5] + [-1], key, g, 9, with_bias)


@pytest.mark.gpu
@pytest.mark.parametrize("t,e,groups,top", [(300, 64, 32, 9), (300, 60, 20, 7), (2100, 256, 64, 17), (2100, 120, 40, 11),
                                            (2100, 256, 32, 16), (2100, 192, 48, 47), (2100, 102, 17, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_scores_next_to_each_other(t, e, groups, top, score, with_bias):
    """All of a token's experts within a few steps of fp32, empty groups and masked experts among them."""
    gen = torch.Generator().manual_seed(e + t)
    x = torch.randn(t, 1, generator=gen).expand(t, e).contiguous()
    x = x * (1.0 + torch.randint(-3, 4, (t, e), generator=gen) * 2.0 ** -22)
    x[1::4] = torch.where(torch.rand(x[1::4].shape, generator=gen) < 0.9, -INF, x[1::4])
    x[2::4, :e // groups] = -INF
    x[3::4] += torch.rand(x[3::4].shape, generator=gen) * 1e-5
    bias = 0.25 + torch.randint(-4, 5, (e,), generator=gen) * 2.0 ** -24 if with_bias else None
    for best in (1, 2):
        check(x, 6, groups, top, best, score, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("t,e,groups,top", [(300, 64, 32, 9), (301, 60, 20, 7), (2101, 256, 64, 17), (2100, 120, 40, 11), (33, 36, 18, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_choice_and_ties(t, e, groups, top, score, best, with_bias):
    """Clear scores, and groups and experts of equal ones: the lowest index first, exactly."""
    gen = torch.Generator().manual_seed(e + t + best)
    x = torch.randn(t, e, generator=gen) * 1.5
    x[1::3] = torch.randint(-2, 3, x[1::3].shape, generator=gen).float() * 0.5
    x[2::9] = 0.0
    x[4::9, e // 2:] = -INF
    bias = torch.randint(-1, 2, (e,), generator=gen).float() * 0.25 if with_bias else None
    check(x, min(6, top * (e // groups)), groups, top, best, score, bias, exact=best == 1)
