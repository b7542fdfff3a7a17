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


def dz_of(dy, c, act):
    """dz = dy act'(c) by the formulas, float64."""
    if act == "none":
        return dy
    if act == "swiglu":
        v, d = c.reshape(c.shape[0], -1, 2, 32), dy.reshape(dy.shape[0], -1, 32)
        x, g = v[:, :, 0], v[:, :, 1]
        s = torch.sigmoid(g)
        return torch.stack([d * g * s, d * x * (s + g * s * (1 - s))], 2).reshape(c.shape)
    if act == "srelu":
        return dy * 2.0 * c.clamp(min=0.0)
    u = 2.0 * ref.C * (c + ref.A * c ** 3)
    s = torch.sigmoid(u)
    return dy * (s + c * s * (1 - s) * 2.0 * ref.C * (1 + 3 * ref.A * c * c))


def check_backward(m, n, k, act, groups, dw_dtype):
    x, w, _, off, gen = make(m, n, k, groups, m + n + 1)
    n_out = n // 2 if act == "swiglu" else n
    dy = torch.randn(m, n_out, generator=gen).to(torch.bfloat16)
    dy[dy == 0] = 0.5
    c = (torch.randn(m, n, generator=gen) * 2).to(torch.bfloat16)
    clean = c.clone()
    spots = [(0, 5), (m // 2, n - 1), (m - 1, n - 40)]
    for i, j in spots:
        c[i, j] = math.nan
        clean[i, j] = 0.0
    print(f"[gpu-case] linear backward NaN m={m} n={n} k={k} {act} groups={groups} {dw_dtype}", flush=True)
    got = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), c=c.cuda(), act=act, offsets=None if off is None else off.cuda(),
                             dw_dtype=dw_dtype)
    want = ref.linear_backward(dy, x, w, clean, act, off)
    lost = torch.isnan(dz_of(dy.double(), c.double(), act))
    assert lost.any()
    group = torch.zeros(m, dtype=torch.long) if off is None else torch.searchsorted(off.long(), torch.arange(m), right=True)
    bad_db = torch.zeros(max(groups, 1), n, dtype=torch.bool)
    for i, j in lost.nonzero().tolist():
        bad_db[group[i], j] = True
    # a NaN of dz reaches its row of dx, its row of dw and its entry of db
    masks = {"dx": lost.any(1)[:, None].expand(m, k), "dw": bad_db[:, :, None].expand(-1, n, k).reshape(w.shape),
             "db": bad_db.reshape(w.shape[:-1])}
    for name, g in zip(("dx", "dw", "db"), got):
        r, bound = want[name]
        g, nan = g.cpu().double(), masks[name]
        assert torch.equal(torch.isnan(g), nan), (name, int(torch.isnan(g).sum()), int(nan.sum()))
        eps = ref.F32 if name == "db" or (name == "dw" and dw_dtype == "f32") else ref.BF16
        bad = (g - r)[~nan].abs() > (bound * (1 + eps) + eps * r.abs() + 1e-38)[~nan]
        assert not bad.any(), (name, int(bad.sum()))


@pytest.mark.parametrize("act", ["swiglu", "srelu"])
@pytest.mark.parametrize("m,n,k,groups", [(5, 320, 200, 0), (300, 256, 1032, 0), (2100, 512, 512, 0), (20, 128, 256, 16),
                                          (2000, 512, 328, 3)])
def test_backward_keeps_nan(m, n, k, groups, act):
    check_backward(m, n, k, act, groups, "f32" if m % 3 else "bf16")


@pytest.mark.parametrize("m,n,k,groups", [(5, 320, 200, 0), (300, 256, 1032, 0), (2100, 512, 512, 0), (20, 128, 256, 16),
                                          (2000, 512, 328, 3)])
def test_gelu_backward_keeps_nan(m, n, k, groups):
    check_backward(m, n, k, "gelu", groups, "f32" if m % 3 else "bf16")
