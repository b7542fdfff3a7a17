"""GPU tests of linear and its gradients against the float64 reference.
Every bound is the one derived in layer_ref."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

ACTS = ["none", "swiglu", "srelu", "gelu"]


def make(m, n, k, act, groups, seed, residual=False, empty=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=gen).to(torch.bfloat16)
    w = (torch.randn(*((groups, n, k) if groups else (n, k)), generator=gen) / math.sqrt(k)).to(torch.bfloat16)
    b = torch.randn(*((groups, n) if groups else (n,)), generator=gen) * 0.3
    off = None
    if groups:
        cut = torch.sort(torch.randint(0, m + 1, (groups,), generator=gen)).values
        cut[-1] = m
        if empty and groups > 2:
            cut[1] = cut[0]
        off = torch.sort(cut).values.to(torch.int32)
    n_out = n // 2 if act == "swiglu" else n
    res = torch.randn(m, n_out, generator=gen).to(torch.bfloat16) if residual else None
    return x, w, b, off, res, gen


def cuda(t):
    return None if t is None else t.cuda()


def check_forward(m, n, k, act, groups, seed=1, residual=False, bias=True, dtype="bf16"):
    x, w, b, off, res, _ = make(m, n, k, act, groups, seed, residual)
    b = b if bias else None
    print(f"[gpu-case] linear m={m} n={n} k={k} {act} groups={groups} residual={residual} {dtype}", flush=True)
    y, c = mg.linear(x.cuda(), w.cuda(), bias=cuda(b), act=act, residual=cuda(res), offsets=cuda(off), save_c=True,
                     dtype=dtype)
    y2 = mg.linear(x.cuda(), w.cuda(), bias=cuda(b), act=act, residual=cuda(res), offsets=cuda(off), dtype=dtype)
    assert torch.equal(y, y2)
    r, z, mag = ref.linear(x, w, b, act, res, off)
    zb = (k + 8) * ref.F32 * mag
    assert ((c.cpu().double() - z).abs() <= zb * 1.01 + ref.BF16 * z.abs()).all()
    bound = ref.linear_bound(z, mag, k, act, res, ref.BF16 if dtype == "bf16" else ref.F32)
    bad = (y.cpu().double() - r).abs() > bound
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4])


SHAPES = [(1, 64, 8), (1, 2816, 2048), (3, 128, 72), (5, 192, 1408), (16, 64, 264), (17, 320, 512), (33, 64, 2048),
          (64, 256, 64), (100, 192, 136), (129, 1408, 200), (257, 320, 1000), (300, 576, 2056), (512, 512, 512)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward(m, n, k, act):
    check_forward(m, n, k, act, 0, seed=m + n)


@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (4, 24, 16), (40, 8, 2048), (130, 72, 1032), (260, 264, 328), (700, 1000, 504)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_odd_widths(m, n, k, dtype):
    check_forward(m, n, k, "none", 0, dtype=dtype)
    check_forward(m, n, k, "gelu", 0, dtype=dtype, residual=True, bias=False)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_residual(act, dtype):
    for m, n, k in [(1, 128, 512), (19, 256, 264), (200, 320, 264), (600, 512, 320)]:
        check_forward(m, n, k, act, 0, residual=True, dtype=dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,groups", [(1, 64, 64, 3), (6, 128, 256, 64), (96, 192, 264, 64), (50, 64, 72, 1000),
                                          (300, 320, 136, 5), (1000, 512, 512, 7), (2000, 192, 328, 64), (600, 256, 64, 1)])
def test_forward_grouped(m, n, k, groups, act):
    check_forward(m, n, k, act, groups, seed=m + groups, residual=groups % 2 == 1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,dtype", [(4097, "bf16"), (4099, "f32"), (4112, "bf16"), (4113, "bf16")])
def test_forward_few_rows_past_whole_tiles(m, act, dtype):
    """A handful of rows behind whole tiles (up to 16 go by the kernel for few rows)."""
    check_forward(m, 2048, 200, act, 0, seed=m, residual=True, dtype=dtype)


def test_forward_long_sums():
    for m in (2, 40, 300):
        check_forward(m, 64, 16384, "none", 0)


@pytest.mark.parametrize("m,n,k", [(4096, 2816, 2048), (16384, 64, 2048), (3000, 2048, 1408), (2500, 2560, 520)])
def test_forward_large(m, n, k):
    """Large products: against an fp64 product on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    b = torch.randn(n, generator=gen, device="cuda")
    print(f"[gpu-case] linear large m={m} n={n} k={k}", flush=True)
    for dtype, eps in (("bf16", ref.BF16), ("f32", ref.F32)):
        y = mg.linear(x, w, bias=b, dtype=dtype)
        z = x.double() @ w.double().t() + b.double()
        mag = x.double().abs() @ w.double().abs().t() + b.double().abs()
        assert ((y.double() - z).abs() <= (k + 8) * ref.F32 * mag + eps * z.abs()).all()


def check_backward(m, n, k, act, groups, seed=1, dw_dtype="bf16", need=("dx", "dw", "db")):
    x, w, _, off, _, gen = make(m, n, k, act, groups, seed)
    n_out = n // 2 if act == "swiglu" else n
    dy = torch.randn(m, n_out, generator=gen).to(torch.bfloat16)
    c = (torch.randn(m, n, generator=gen) * 2).to(torch.bfloat16) if act != "none" else None
    print(f"[gpu-case] linear backward m={m} n={n} k={k} {act} groups={groups} {dw_dtype} {need}", flush=True)
    got = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), c=cuda(c), act=act, offsets=cuda(off), need=need,
                             dw_dtype=dw_dtype)
    want = ref.linear_backward(dy, x, w, c, act, off)
    for name, g in zip(("dx", "dw", "db"), got):
        assert (g is None) == (name not in need)
        if g is None:
            continue
        r, bound = want[name]
        eps = ref.F32 if name == "db" or (name == "dw" and dw_dtype == "f32") else ref.BF16
        bad = (g.cpu().double() - r).abs() > bound * (1 + eps) + eps * r.abs() + 1e-38
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4])
    return got


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 64, 8), (2, 192, 264), (17, 64, 2048), (100, 320, 136), (129, 1408, 200),
                                   (300, 576, 1032), (600, 512, 512)])
def test_backward(m, n, k, act):
    check_backward(m, n, k, act, 0, seed=m + k)


@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (5, 24, 16), (70, 8, 1032), (333, 72, 264), (700, 1000, 504)])
def test_backward_odd_widths(m, n, k):
    check_backward(m, n, k, "none", 0, dw_dtype="f32")
    check_backward(m, n, k, "gelu", 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,groups", [(1, 64, 64, 3), (6, 128, 256, 64), (96, 192, 264, 64), (300, 320, 136, 5),
                                          (1000, 512, 512, 7), (2000, 192, 328, 64), (40, 64, 8, 300)])
def test_backward_grouped(m, n, k, groups, act):
    check_backward(m, n, k, act, groups, seed=m + groups, dw_dtype="f32" if groups == 5 else "bf16")


@pytest.mark.parametrize("need", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_backward_parts(need, act):
    check_backward(150, 192, 136, act, 0, need=need)
    check_backward(150, 192, 136, act, 4, need=need)


def test_backward_long_sums():
    """Weight gradients over many rows (the sum is split and joined)."""
    check_backward(30011, 64, 72, "none", 0, dw_dtype="f32")
    check_backward(30011, 64, 72, "swiglu", 3)


@pytest.mark.parametrize("m,n,k", [(4096, 2816, 2048), (8000, 2048, 1408)])
def test_backward_large(m, n, k):
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    dy = torch.randn(m, n, generator=gen, device="cuda").to(torch.bfloat16)
    print(f"[gpu-case] linear backward large m={m} n={n} k={k}", flush=True)
    dx, dw, db = mg.linear_backward(dy, x, w, dw_dtype="f32")
    d, xd, wd = dy.double(), x.double(), w.double()
    for g, r, mag, terms, eps in ((dx, d @ wd, d.abs() @ wd.abs(), n, ref.BF16), (dw, d.t() @ xd, d.abs().t() @ xd.abs(), m, ref.F32),
                                  (db, d.sum(0), d.abs().sum(0), m, ref.F32)):
        assert ((g.double() - r).abs() <= (terms + 8) * ref.F32 * mag + eps * r.abs()).all()


def test_rows_behind_the_last_group():
    """They are neither written nor read."""
    m, n, k, groups = 200, 128, 64, 3
    x, w, b, _, _, gen = make(m, n, k, "none", groups, 5)
    off = torch.tensor([40, 40, 150], dtype=torch.int32)
    x[150:] = math.nan
    dy = torch.randn(m, n, generator=gen).to(torch.bfloat16)
    dy[150:] = math.nan
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    y = mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), offsets=off.cuda(), out=out)
    assert (y[150:] == 7.0).all() and torch.isfinite(y[:150]).all()
    dx, dw, db = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), offsets=off.cuda())
    assert torch.isfinite(dx[:150]).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
    assert (dw[1] == 0).all() and (db[1] == 0).all()              # the empty group


def test_neighbours_do_not_leak():
    """A group's infinities and NaN stay in its own rows and gradients."""
    m, n, k, groups = 300, 128, 136, 4
    x, w, b, _, _, gen = make(m, n, k, "none", groups, 6)
    off = torch.tensor([70, 133, 222, 300], dtype=torch.int32)
    dy = torch.randn(m, n, generator=gen).to(torch.bfloat16)
    x[70:133], w[1], dy[70:133] = math.inf, math.nan, math.nan
    y = mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), offsets=off.cuda())
    rest = torch.cat([torch.arange(70), torch.arange(133, 300)])
    assert torch.isfinite(y[rest.cuda()]).all() and torch.isnan(y[70:133]).all()
    dx, dw, db = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), offsets=off.cuda())
    assert torch.isfinite(dx[rest.cuda()]).all()
    for g in (0, 2, 3):
        assert torch.isfinite(dw[g]).all() and torch.isfinite(db[g]).all()


def test_foreign_offsets_stay_inside():
    """Offsets that decrease or leave the rows address nothing outside them."""
    m, n, k, groups = 100, 64, 64, 5
    x, w, b, _, _, gen = make(m, n, k, "none", groups, 7)
    dy = torch.randn(m, n, generator=gen).to(torch.bfloat16)
    for off in ([50, 20, 90, 60, 100], [-5, 30, 2 ** 31 - 1, 40, 100], [1000, 1000, 1000, 1000, 1000], [-1, -1, -1, -1, -1]):
        o = torch.tensor(off, dtype=torch.int32).cuda()
        y = mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), offsets=o)
        dx, dw, db = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), offsets=o)
        torch.cuda.synchronize()
        assert y.shape == (m, n) and torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_offsets_that_name_rows_many_times():
    """Ends that rise and fall name more row tiles than a launch has: all results
    stay inside, for every kernel (wide, narrow, few rows)."""
    groups = 256
    off = torch.tensor([1000, 0] * (groups // 2), dtype=torch.int32).cuda()
    for m, n, k in ((5000, 320, 200), (5000, 64, 64), (1000, 64, 64), (100, 64, 64)):
        print(f"[gpu-case] linear falling offsets m={m} n={n} k={k}", flush=True)
        x, w, b, _, _, gen = make(m, n, k, "none", groups, 7)
        dy = torch.randn(m, n, generator=gen).to(torch.bfloat16)
        y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
        mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), offsets=off, out=y)
        assert (y[1000:] == 7).all() and torch.isfinite(y).all()
        dx, dw, db = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), offsets=off)
        torch.cuda.synchronize()
        assert torch.isfinite(dw).all() and torch.isfinite(db).all() and (dw[1::2] == 0).all() and (db[1::2] == 0).all()
        # the first group's own rows come first in every count
        d, xd = dy[:1000].double(), x[:1000].double()
        r, mag = d.t() @ xd, d.abs().t() @ xd.abs()
        assert ((dw[0].cpu().double() - r).abs() <= 1008 * ref.F32 * mag + ref.BF16 * r.abs()).all()
        assert ((db[0].cpu().double() - d.sum(0)).abs() <= 1008 * ref.F32 * d.abs().sum(0)).all()


@pytest.mark.parametrize("n,k", [(64, 2048), (2048, 64), (512, 2048)])
def test_more_than_two_to_the_31_elements(n, k):
    """Operands or results whose element numbers pass 32 bits: checked on the
    last rows, and dw over all of them."""
    m = 1100000
    print(f"[gpu-case] linear m={m} n={n} k={k}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(m, k, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    y, c = mg.linear(x, w, act="srelu", save_c=True)
    assert max(x.numel(), y.numel()) > 2 ** 31
    wd = w.double()
    for part in (slice(0, 300), slice(m - 300, m)):
        xd = x[part].double()
        z, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
        assert ((c[part].double() - z).abs() <= (k + 8) * ref.F32 * mag * 1.01 + ref.BF16 * z.abs()).all()
    del y, c
    dy = torch.randn(m, n, generator=gen, device="cuda", dtype=torch.bfloat16)
    dx, dw, db = mg.linear_backward(dy, x, w, dw_dtype="f32")
    for part in (slice(0, 300), slice(m - 300, m)):
        d = dy[part].double()
        r, mag = d @ wd, d.abs() @ wd.abs()
        assert ((dx[part].double() - r).abs() <= (n + 8) * ref.F32 * mag + ref.BF16 * r.abs()).all()
    rows, cols = slice(0, 16), slice(k - 16, k)
    r = torch.zeros(16, 16, dtype=torch.float64, device="cuda")
    mag, s, sa = r.clone(), torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    for at in range(0, m, 100000):
        d, xd = dy[at:at + 100000].double(), x[at:at + 100000, cols].double()
        r += d[:, rows].t() @ xd
        mag += d[:, rows].abs().t() @ xd.abs()
        s += d.sum(0)
        sa += d.abs().sum(0)
    assert ((dw[rows, cols].double() - r).abs() <= (m + 8) * ref.F32 * mag + ref.F32 * r.abs()).all()
    assert ((db.double() - s).abs() <= (m + 8) * ref.F32 * sa).all()


# every kernel of the forward: few rows, the three tiles, parts of r and their join, few rows past whole tiles
PATHS = [(5, 320, 200), (256, 512, 512), (300, 256, 4096), (1100, 1024, 512), (4099, 2048, 200), (8192, 2048, 520)]


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("m,n,k", PATHS)
def test_residual_in_place(m, n, k, act):
    """y may be the residual itself: the same bits as in memory of its own."""
    x, w, b, _, res, _ = make(m, n, k, act, 0, m, residual=True)
    print(f"[gpu-case] linear in place m={m} n={n} k={k} {act}", flush=True)
    want = mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), act=act, residual=res.cuda())
    y = res.cuda()
    assert mg.linear(x.cuda(), w.cuda(), bias=b.cuda(), act=act, residual=y, out=y) is y
    assert torch.equal(y, want)


@pytest.mark.parametrize("m,n,k", PATHS)
def test_captured_calls(m, n, k):
    """Forward and backward in a graph, replayed between eager calls and on new inputs: the eager bits."""
    x, w, b, _, res, gen = make(m, n, k, "swiglu", 0, m, residual=True)
    dy = torch.randn(m, n // 2, generator=gen).to(torch.bfloat16)
    xs = [x.cuda(), x.flip(0).contiguous().cuda(), (x * 0.5).cuda()]
    w, b, res, dy = w.cuda(), b.cuda(), res.cuda(), dy.cuda()
    print(f"[gpu-case] linear captured m={m} n={n} k={k}", flush=True)

    def run(x):
        y, c = mg.linear(x, w, bias=b, act="swiglu", residual=res, save_c=True)
        return (y, c, *mg.linear_backward(dy, x, w, c=c, act="swiglu"))
    held = xs[0].clone()
    run(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(held)
    for x in xs:
        held.copy_(x)
        graph.replay()
        want = run(x)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_activation_extremes():
    """Pre-activations from -1e30 to 1e30 give the activation's limits, no NaN."""
    for act in ("gelu", "swiglu", "srelu"):
        v = torch.tensor([-1e30, -1e4, -50.0, -1.0, 0.0, 1.0, 50.0, 1e4], dtype=torch.float32)
        x = v.to(torch.bfloat16).reshape(-1, 1).repeat(1, 8)
        x[:, 1:] = 0
        w = torch.zeros(64, 8, dtype=torch.bfloat16)
        w[:, 0] = 1
        y, c = mg.linear(x.cuda(), w.cuda(), act=act, save_c=True, dtype="f32")
        r = ref.act(x[:, :1].double().repeat(1, 64), act)
        assert torch.allclose(y.cpu().double(), r.clamp(max=3.4028234e38), rtol=1e-5, atol=1e-30)
        dy = torch.ones(8, y.shape[1], dtype=torch.bfloat16)
        dx, dw, db = mg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), c=c, act=act)
        fine = slice(1, None) if act != "srelu" else slice(0, None)
        assert torch.isfinite(dx.float()[fine]).all() and torch.isfinite(db[0])


def test_empty_rows():
    w = torch.randn(3, 64, 64, device="cuda").to(torch.bfloat16)
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert mg.linear(x, w, offsets=off).shape == (0, 64)
    dx, dw, db = mg.linear_backward(x, x, w, offsets=off)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
