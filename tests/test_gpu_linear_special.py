"""linear and its gradients on NaN and infinities: what the formulas give, in
the rows and columns that they reach and nowhere else, on every kernel."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ["none", "swiglu", "srelu", "gelu"]
# every kernel of the forward: few rows, the three tiles, parts of r and their join, few rows past whole tiles
PATHS = [(5, 320, 200), (256, 512, 512), (300, 256, 4096), (1100, 1024, 512), (4099, 2048, 200), (8192, 2048, 520)]
# and with groups: few rows, narrow and wide tiles
GROUPED = [(20, 128, 256, 16), (300, 320, 136, 5), (2000, 512, 328, 3)]


def make(m, n, k, groups, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=gen).to(torch.bfloat16)
    w = (torch.randn(*((groups, n, k) if groups else (n, k)), generator=gen) / math.sqrt(k)).to(torch.bfloat16)
    w[w == 0] = 0.5                                      # (0 times an infinity is not what is looked at)
    b = torch.randn(*((groups, n) if groups else (n,)), generator=gen) * 0.3
    off = None
    if groups:
        off = (torch.arange(1, groups + 1) * m // groups).to(torch.int32)
    return x, w, b, off, gen


def agree(got, want, bound):
    """NaN where the formula has NaN, its infinities, and finite numbers within the bound."""
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (int(torch.isnan(got).sum()), int(torch.isnan(want).sum()))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    fine = torch.isfinite(want)
    # (a bound that is no number belongs to a row or column that holds an infinity: its finite values are exact)
    bound = torch.where(torch.isfinite(bound), bound, 0.0)
    bad = (got - want)[fine].abs() > bound[fine]
    assert not bad.any(), int(bad.sum())


def check_forward(m, n, k, act, groups, dtype):
    x, w, b, off, _ = make(m, n, k, groups, m + n)
    last = m - 1                                         # (where few rows follow whole tiles: one of them)
    x[0, 3] = math.nan
    if m > 3:
        x[m // 2, k - 1], x[m // 3, 0] = math.inf, -math.inf
    x[last, k // 2] = math.nan
    b.reshape(-1, n)[-1, 7] = math.nan
    print(f"[gpu-case] linear NaN m={m} n={n} k={k} {act} groups={groups} {dtype}", flush=True)
    y, c = mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), act=act, offsets=None if off is None else off.cuda(), save_c=True,
                     dtype=dtype)
    r, z, mag = ref.linear(x, w, b, act, None, off)
    agree(c, z, (k + 8) * ref.F32 * mag * 1.01 + ref.BF16 * z.abs())
    eps = ref.BF16 if dtype == "bf16" else ref.F32
    agree(y, r, ref.linear_bound(z, mag, k, act, None, eps))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", PATHS)
def test_forward_keeps_nan_and_infinities(m, n, k, act):
    check_forward(m, n, k, act, 0, "bf16" if m % 2 else "f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,groups", GROUPED)
def test_grouped_forward_keeps_nan_and_infinities(m, n, k, groups, act):
    check_forward(m, n, k, act, groups, "bf16")
