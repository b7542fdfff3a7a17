"""GPU tests of rows kept in 8 bits: quantise and dequantise, linear that keeps
c so, and its gradients from x and c in 8 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref  # noqa: E402
import more_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FMTS = ["e4m3", "e5m2"]


def cuda(t):
    return None if t is None else t.cuda()


def planes(byte):
    return byte.reshape(byte.shape[0], -1, 4).transpose(0, 1).contiguous()


def plain_zero(codes):
    """Negative zeros as zeros."""
    return np.where((codes & 0x7F) == 0, 0, codes)


# ---- rows ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layout", ["row_major", "kplanes"])
@pytest.mark.parametrize("kind", [BF, torch.float32])
@pytest.mark.parametrize("t,h", [(1, 128), (3, 256), (5, 1152), (33, 640), (129, 2048), (1000, 384)])
def test_quantise(t, h, fmt, layout, kind):
    check_quantise(t, h, fmt, layout, kind)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t,h", [(1, 32), (1, 96), (7, 32), (5, 160), (127, 224), (513, 32), (3, 1056)])
def test_quantise_odd_widths(t, h, fmt):
    check_quantise(t, h, fmt, "row_major", BF)
    check_quantise(t, h, fmt, "row_major", torch.float32)


def check_quantise(t, h, fmt, layout, kind):
    gen = torch.Generator().manual_seed(t + h)
    x = (torch.randn(t, h, generator=gen) * torch.exp(3 * torch.randn(t, h // 32, generator=gen)).repeat_interleave(32, 1)).to(kind)
    x[0, :32] = 0
    print(f"[gpu-case] quantise {t}x{h} {fmt} {layout} {kind}", flush=True)
    codes, sf = mg.quantise(x.cuda(), dtype=fmt, sf_layout=layout)
    wc, ws = ref.mx_encode(x.double(), fmt)
    assert np.array_equal(ref.rowmajor(sf.cpu(), layout).numpy(), ws)
    assert np.array_equal(plain_zero(codes.cpu().numpy()), plain_zero(wc))
    want = ref.decode(codes.cpu(), torch.from_numpy(ws), fmt)
    for to, name in ((torch.float32, "f32"), (BF, "bf16")):
        back = mg.dequantise((codes, sf), dtype=fmt, sf_layout=layout, to=name)
        assert back.dtype is to and torch.equal(back.cpu(), want.to(to))
    marked = torch.full_like(codes, 0x5A), torch.full_like(sf, 0x5A)
    got = mg.quantise(x.cuda(), dtype=fmt, sf_layout=layout, out=marked)
    assert got[0] is marked[0] and torch.equal(got[0], codes) and torch.equal(got[1], sf)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_and_scale(fmt):
    """All 256 codes under every scale byte: what they stand for, in fp32 and BF16."""
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 256).repeat(256, 1)
    byte = torch.arange(256, dtype=torch.uint8).reshape(256, 1).repeat(1, 8)
    want = ref.decode(codes, byte, fmt)
    bad = {"e4m3": (codes & 0x7F) == 0x7F, "e5m2": (codes & 0x7F) > 0x7C}[fmt]      # NaN codes
    inf = (codes & 0x7F) == 0x7C if fmt == "e5m2" else torch.zeros_like(bad)
    for to, name in ((torch.float32, "f32"), (BF, "bf16")):
        got = mg.dequantise((codes.cuda(), byte.cuda()), dtype=fmt, to=name).cpu()
        w = want.to(torch.float32).to(to)
        ok = ~bad & ~inf & (byte.repeat_interleave(32, 1) < 255)
        assert torch.equal(got[ok], w[ok])
        assert torch.isnan(got[bad | (byte.repeat_interleave(32, 1) == 255)]).all()
        fine = inf & (byte.repeat_interleave(32, 1) < 255)
        assert torch.isinf(got[fine]).all()


@pytest.mark.parametrize("kind", [BF, torch.float32])
def test_quantise_edges(kind):
    """Blocks on both sides of a scale's border, subnormal, huge, infinite and NaN."""
    rows = []
    for q in (448.0, 57344.0):
        for p in (-120, -20, -1, 0, 1, 40, 100):
            for f in (1.0, 1.0 + 2.0 ** -7, 1.0 - 2.0 ** -8):
                v = torch.zeros(32, dtype=torch.float64)
                v[7], v[9] = q * 2.0 ** p * f, -q * 2.0 ** (p - 3) / 3
                rows.append(v if v.abs().max() < 3e38 else v * 0)
    x = torch.stack(rows).to(kind)
    x[0, 3], x[1, 4], x[2, 5] = math.nan, math.inf, -math.inf
    x[3] = torch.finfo(kind).max
    x[4] = 2.0 ** -126
    x[5] = 2.0 ** -133
    for fmt in FMTS:
        codes, sf = mg.quantise(x.cuda(), dtype=fmt)
        wc, ws = ref.mx_encode(x.double(), fmt)
        assert np.array_equal(sf.cpu().numpy(), ws)
        assert np.array_equal(plain_zero(codes.cpu().numpy()), plain_zero(wc))
        assert torch.isnan(mg.dequantise((codes, sf), dtype=fmt)[:3]).all()


def test_dispatch_writes_the_same_rows():
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(70, 512, generator=gen).to(BF).cuda()
    plan = mg.sort_tokens(torch.zeros(70, 1, dtype=torch.int32, device="cuda"), 1, m_aligned=1)
    for layout in ("row_major", "kplanes"):
        a = mg.dispatch(x, plan, dtype="e4m3", sf_layout=layout)
        b = mg.quantise(x, sf_layout=layout)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_past_32_bits():
    t, h = (1 << 20) + 1, 2080
    x = torch.zeros(t, h, dtype=BF, device="cuda")
    x[-1] = torch.arange(h, device="cuda").remainder(9).to(BF)
    codes, sf = mg.quantise(x)
    wc, ws = ref.mx_encode(x[-1:].cpu().double(), "e4m3")
    assert np.array_equal(sf[-1:].cpu().numpy(), ws) and np.array_equal(codes[-1:].cpu().numpy(), wc)
    assert torch.equal(mg.dequantise((codes, sf))[-1], x[-1])
    assert not codes[:-1].any()


def test_no_rows():
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    codes, sf = mg.quantise(e)
    assert codes.shape == (0, 64) and sf.shape == (0, 2) and mg.dequantise((codes, sf)).shape == (0, 64)


# ---- linear that keeps c -------------------------------------------------------------

def make(m, n, k, act, groups, seed, residual=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=gen).to(BF)
    w = (torch.randn(*((groups, n, k) if groups else (n, k)), generator=gen) / math.sqrt(k)).to(BF)
    b = torch.randn(*((groups, n) if groups else (n,)), generator=gen) * 0.3
    off = None
    if groups:
        cut = torch.sort(torch.randint(0, m + 1, (groups,), generator=gen)).values
        cut[-1] = m
        if groups > 2:
            cut[1] = cut[0]
        off = torch.sort(cut).values.to(torch.int32)
    n_out = n // 2 if act == "swiglu" else n
    res = torch.randn(m, n_out, generator=gen).to(BF) if residual else None
    return x, w, b, off, res, gen


def check_forward(m, n, k, act, groups, fmt="e4m3", seed=1, residual=False, bias=True, dtype="bf16"):
    x, w, b, off, res, _ = make(m, n, k, act, groups, seed, residual)
    b = b if bias else None
    print(f"[gpu-case] linear keeps {fmt} m={m} n={n} k={k} {act} groups={groups} residual={residual} {dtype}", flush=True)
    y, (codes, sf) = mg.linear(x.cuda(), w.cuda(), bias=cuda(b), act=act, residual=cuda(res), offsets=cuda(off), save_c=fmt,
                               dtype=dtype)
    r, z, mag = layer_ref.linear(x, w, b, act, res, off)
    off_z = (k + 8) * ref.F32 * mag
    ref.check_mx(codes, sf, fmt, z, off_z)
    bound = layer_ref.linear_bound(z, mag, k, act, res, ref.BF16 if dtype == "bf16" else ref.F32)
    assert not ((y.cpu().double() - r).abs() > bound).any()


SHAPES = [(1, 64, 8), (1, 2816, 2048), (3, 128, 72), (5, 192, 1408), (16, 64, 264), (17, 320, 512), (33, 64, 2048),
          (100, 192, 136), (129, 1408, 200), (257, 320, 1000), (300, 576, 2056), (512, 512, 512), (2050, 2048, 136)]


@pytest.mark.parametrize("act", ["none", "swiglu", "srelu", "gelu"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward(m, n, k, act):
    check_forward(m, n, k, act, 0, seed=m + n)


@pytest.mark.parametrize("m,n,k", [(1, 32, 8), (40, 96, 2048), (130, 352, 1032), (700, 1056, 504), (300, 160, 4096), (2000, 2080, 64)])
@pytest.mark.parametrize("fmt", FMTS)
def test_forward_odd_widths(m, n, k, fmt):
    check_forward(m, n, k, "none", 0, fmt, dtype="f32")
    check_forward(m, n, k, "gelu", 0, fmt, residual=True, bias=False)


@pytest.mark.parametrize("act", ["none", "swiglu", "srelu", "gelu"])
@pytest.mark.parametrize("m,n,k,groups", [(1, 64, 64, 3), (6, 128, 256, 64), (96, 192, 264, 64), (50, 64, 72, 1000),
                                          (300, 320, 136, 5), (1000, 512, 512, 7), (2000, 192, 328, 64), (600, 256, 64, 1)])
def test_forward_grouped(m, n, k, groups, act):
    check_forward(m, n, k, act, groups, FMTS[m % 2], seed=m + groups, residual=groups % 2 == 1)


@pytest.mark.parametrize("m,n,k", [(4096, 2816, 2048), (3000, 2048, 1408)])
def test_forward_large(m, n, k):
    """Tiles of 256 x 256, whole and split: c as its BF16 form says, and y bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=gen, device="cuda").to(BF)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(BF)
    y0, c0 = mg.linear(x, w, act="swiglu", save_c=True)
    y, (codes, sf) = mg.linear(x, w, act="swiglu", save_c="e4m3")
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    ref.check_mx(codes, sf, "e4m3", z.cpu(), (k + 8) * ref.F32 * mag.cpu())
    bound = layer_ref.linear_bound(z.cpu(), mag.cpu(), k, "swiglu", None, ref.BF16)
    assert ((y.double() - y0.double()).abs().cpu() <= 2 * bound).all()


def check_on_gpu(m, n, k, act, groups, fmt):
    """c against float64 products on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.randn(m, k, generator=gen, device="cuda").to(BF)
    w = (torch.randn(max(groups, 1), n, k, generator=gen, device="cuda") / math.sqrt(k)).to(BF)
    b = torch.randn(max(groups, 1), n, generator=gen, device="cuda") * 0.3
    ends = [m]
    if groups:
        ends = torch.sort(torch.randint(0, m + 1, (groups - 1,), generator=gen, device="cuda")).values.tolist() + [m]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda") if groups else None
    print(f"[gpu-case] linear keeps {fmt} m={m} n={n} k={k} {act} groups={groups}", flush=True)
    if groups:
        y, (codes, sf) = mg.linear(x, w, bias=b, act=act, offsets=off, save_c=fmt)
        y0, _ = mg.linear(x, w, bias=b, act=act, offsets=off, save_c=True)
    else:
        y, (codes, sf) = mg.linear(x, w[0], bias=b[0], act=act, save_c=fmt)
        y0, _ = mg.linear(x, w[0], bias=b[0], act=act, save_c=True)
    z, mag, at = torch.empty(m, n, dtype=torch.float64), torch.empty(m, n, dtype=torch.float64), 0
    for g, end in enumerate(ends):
        xs, ws = x[at:end].double(), w[g].double()
        z[at:end] = (xs @ ws.t() + b[g].double()).cpu()
        mag[at:end] = (xs.abs() @ ws.abs().t() + b[g].double().abs()).cpu()
        at = end
    ref.check_mx(codes, sf, fmt, z, (k + 8) * ref.F32 * mag)
    bound = layer_ref.linear_bound(z, mag, k, act, None, ref.BF16)
    assert ((y.cpu().double() - y0.cpu().double()).abs() <= 2 * bound).all()


@pytest.mark.parametrize("m,n,k,act,fmt", [(300, 160, 4096, "none", "e5m2"), (600, 1056, 8192, "gelu", "e4m3"),
                                           (300, 2048, 8192, "swiglu", "e4m3"), (2500, 2048, 8192, "swiglu", "e5m2"),
                                           (700, 512, 16384, "srelu", "e4m3")])
def test_forward_parts_of_r(m, n, k, act, fmt):
    """Sums split among workgroups: the join keeps c."""
    code = {"none": 0, "swiglu": 1, "srelu": 2, "gelu": 7}[act]
    assert mg._load().moegg_linear_saving_workspace(mg.moegg_linear_problem(m, n, k, 1, code, 3), mg.moegg_linear_saved(3, 0, 1)) > 0
    check_on_gpu(m, n, k, act, 0, fmt)


@pytest.mark.parametrize("m,n,k,act,groups,fmt", [(5000, 2048, 520, "swiglu", 6, "e4m3"), (3001, 1056, 2048, "gelu", 20, "e5m2"),
                                                  (777, 2816, 264, "srelu", 64, "e4m3")])
def test_forward_large_grouped(m, n, k, act, groups, fmt):
    check_on_gpu(m, n, k, act, groups, fmt)


def test_rows_behind_the_last_group_are_left():
    x, w, b, _, _, _ = make(300, 128, 64, "gelu", 3, 1)
    off = torch.tensor([100, 100, 170], dtype=torch.int32).cuda()
    lib, u8 = mg._load(), torch.uint8
    c, sf = torch.full((300, 128), 0x5A, dtype=u8, device="cuda"), torch.full((300, 4), 0x5A, dtype=u8, device="cuda")
    y = torch.full((300, 128), 7.0, dtype=BF, device="cuda")
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    p, keep = mg.moegg_linear_problem(300, 128, 64, 3, 7, 3), mg.moegg_linear_saved(3, 0, 1, 0, None, sf.data_ptr())
    need = lib.moegg_linear_saving_workspace(p, keep)
    ws = torch.empty(max(need, 16), dtype=u8, device="cuda")
    a = mg.moegg_linear_args(x.data_ptr(), w.data_ptr(), b.data_ptr(), None, off.data_ptr(), y.data_ptr(), c.data_ptr(), None,
                             None, None, None, ws.data_ptr(), need)
    assert lib.moegg_linear_saving(p, a, keep, torch.cuda.current_stream().cuda_stream) == 0
    assert (c[170:] == 0x5A).all() and (sf[170:] == 0x5A).all() and (y[170:] == 7.0).all()
    _, z, mag = layer_ref.linear(x[:170].cpu(), w.cpu(), b.cpu(), "gelu", None, off.cpu())
    ref.check_mx(c[:170], sf[:170], "e4m3", z, 72 * ref.F32 * mag)


def test_not_numbers_in_c():
    """A block of z with a NaN or an infinity: codes 0 and scale byte 255, NaN when read back."""
    x = torch.ones(40, 64, dtype=BF)
    w = torch.full((128, 64), 0.125, dtype=BF)
    b = torch.zeros(128)
    b[3], b[40], b[100] = math.nan, math.inf, -math.inf
    for m in (1, 40):
        for n, split in ((128, False), (32, True)):
            kk = 4096 if split else 64
            xs, ws = torch.ones(m, kk, dtype=BF).cuda(), torch.full((n, kk), 0.125, dtype=BF).cuda()
            _, (codes, sf) = mg.linear(xs, ws, bias=b[:n].cuda(), save_c="e5m2")
            assert (sf[:, 0] == 255).all() and (codes[:, :32] == 0).all()
            if n == 128:
                assert (sf[:, [1, 3]] == 255).all() and (sf[:, 2] < 255).all()


# ---- gradients ---------------------------------------------------------------------

def check_backward(m, n, k, act, groups, fmt="e4m3", layout="row_major", seed=1, need=("dx", "dw", "db"), dw_dtype="bf16",
                   both=True):
    """The gradients of the values that the codes stand for: those of linear_backward() from the same
    values in BF16 bit for bit, and within the derived bounds of the float64 ones."""
    _, w, _, off, _, gen = make(m, n, k, act, groups, seed)
    dy = torch.randn(m, n // 2 if act == "swiglu" else n, generator=gen).to(BF)
    print(f"[gpu-case] linear backward from {fmt} m={m} n={n} k={k} {act} groups={groups} {layout} {need} {dw_dtype}", flush=True)
    xc, xs = ref.mx_encode(torch.randn(m, k, generator=gen).double(), fmt)
    cc, cs = ref.mx_encode(2 * torch.randn(m, n, generator=gen).double(), fmt)
    xv, cv = ref.decode(xc, xs, fmt), ref.decode(cc, cs, fmt)
    xs = torch.from_numpy(xs)
    x8 = torch.from_numpy(xc).cuda(), (planes(xs) if layout == "kplanes" else xs).cuda()
    c8 = torch.from_numpy(cc).cuda(), torch.from_numpy(cs).cuda()
    x16, c16 = xv.to(BF), cv.to(BF)
    assert torch.equal(x16.double(), xv) and torch.equal(c16.double(), cv)
    if act == "none":
        c8 = c16 = None
    kw = dict(act=act, offsets=cuda(off), need=need, dw_dtype=dw_dtype)
    how8 = dict(x_dtype=fmt, c_dtype=fmt, sf_layout=layout)
    got = mg.linear_backward(dy.cuda(), x8, w.cuda(), c=c8, **kw, **how8)
    same = mg.linear_backward(dy.cuda(), x16.cuda(), w.cuda(), c=cuda(c16), **kw)
    for a, b in zip(got, same):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    if both and c8 is not None:                          # one of the two in 8 bits
        a = mg.linear_backward(dy.cuda(), x8, w.cuda(), c=cuda(c16), **kw, x_dtype=fmt, sf_layout=layout)
        b = mg.linear_backward(dy.cuda(), x16.cuda(), w.cuda(), c=c8, **kw, c_dtype=fmt)
        for one in (a, b):
            assert all(p is q or torch.equal(p, q) for p, q in zip(one, same))
    want = layer_ref.linear_backward(dy, xv, w, cv if c8 else None, act, off)
    for name, g in zip(("dx", "dw", "db"), got):
        if g is None:
            assert name not in need
            continue
        r, bound = want[name]
        eps = ref.F32 if name == "db" or (name == "dw" and dw_dtype == "f32") else ref.BF16
        assert ((g.cpu().double() - r).abs() <= bound * (1 + eps) + eps * r.abs() + 1e-38).all(), name


@pytest.mark.parametrize("act", ["none", "swiglu", "srelu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 32), (1, 192, 128), (3, 128, 96), (17, 320, 512), (100, 192, 160), (129, 1408, 224),
                                   (257, 320, 992), (700, 512, 512)])
def test_backward(m, n, k, act):
    check_backward(m, n, k, act, 0, FMTS[m % 2], seed=m + n)


@pytest.mark.parametrize("act", ["none", "swiglu", "srelu", "gelu"])
@pytest.mark.parametrize("m,n,k,groups", [(1, 64, 128, 3), (96, 192, 256, 64), (300, 320, 128, 5), (1000, 512, 512, 7),
                                          (600, 256, 128, 1)])
def test_backward_grouped(m, n, k, groups, act):
    check_backward(m, n, k, act, groups, FMTS[m % 2], "kplanes", seed=m + groups, dw_dtype="f32")


@pytest.mark.parametrize("need", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")])
def test_backward_parts(need):
    check_backward(150, 128, 256, "gelu", 0, layout="kplanes", need=need)
    check_backward(150, 128, 256, "swiglu", 4, need=need)


@pytest.mark.parametrize("m,n,k", [(4096, 2816, 2048), (2049, 1408, 2048)])
def test_backward_large(m, n, k):
    """Tiles of 256 x 256: bit for bit as from BF16."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x8 = mg.quantise(torch.randn(m, k, generator=gen, device="cuda"))
    c8 = mg.quantise(torch.randn(m, n, generator=gen, device="cuda"), dtype="e5m2")
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(BF)
    dy = torch.randn(m, n // 2, generator=gen, device="cuda").to(BF)
    got = mg.linear_backward(dy, x8, w, c=c8, act="swiglu", x_dtype="e4m3", c_dtype="e5m2")
    same = mg.linear_backward(dy, mg.dequantise(x8), w, c=mg.dequantise(c8, dtype="e5m2"), act="swiglu")
    assert all(torch.equal(a, b) for a, b in zip(got, same))


@pytest.mark.parametrize("m,n,k,groups,fmt,layout", [
    (6000, 2048, 1408, 12, "e4m3", "kplanes"), (3001, 1408, 2048, 16, "e5m2", "row_major"), (24571, 1408, 2048, 64, "e4m3", "kplanes"),
    (700, 2816, 2080, 9, "e4m3", "row_major"), (4099, 2080, 2144, 0, "e5m2", "row_major"), (40, 2048, 2048, 32, "e4m3", "kplanes"),
    (2500, 1056, 1120, 4, "e4m3", "row_major")])
@pytest.mark.parametrize("need", [("dx", "dw", "db"), ("dw",)])
def test_backward_large_grouped(m, n, k, groups, fmt, layout, need):
    """Ragged and empty groups, widths that end inside a tile, rows that end inside a step: bit for bit as from BF16,
    with NaN scales among the rows of other groups."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x8 = mg.quantise(torch.randn(m, k, generator=gen, device="cuda"), dtype=fmt, sf_layout=layout)
    c8 = mg.quantise(torch.randn(m, n, generator=gen, device="cuda"), dtype=fmt)
    w = (torch.randn(*((groups, n, k) if groups else (n, k)), generator=gen, device="cuda") / math.sqrt(k)).to(BF)
    dy = torch.randn(m, n, generator=gen, device="cuda").to(BF)
    off = None
    if groups:
        cut = torch.sort(torch.randint(0, m - 6, (groups,), generator=gen, device="cuda")).values
        cut[1], cut[-1] = cut[0], m - 7                    # an empty group, and rows behind the last
        off = torch.sort(cut).values.to(torch.int32)
        (x8[1][:, -7:] if layout == "kplanes" else x8[1][-7:]).fill_(255)
    print(f"[gpu-case] linear backward from {fmt} large m={m} n={n} k={k} groups={groups} {layout} {need}", flush=True)
    got = mg.linear_backward(dy, x8, w, c=c8, act="gelu", offsets=off, need=need, x_dtype=fmt, c_dtype=fmt, sf_layout=layout)
    x, c = mg.dequantise(x8, dtype=fmt, sf_layout=layout), mg.dequantise(c8, dtype=fmt)
    same = mg.linear_backward(dy, x, w, c=c, act="gelu", offsets=off, need=need)
    for a, b in zip(got, same):
        if a is not None and a.shape == (m, k) and groups:
            a, b = a[:m - 7], b[:m - 7]
        assert (a is None) == (b is None) and (a is None or (torch.equal(a, b) and not torch.isnan(a).any()))


def test_scale_bytes_of_not_numbers():
    """A scale byte of 255 in x or c: NaN in the gradients that read it, and in no other."""
    gen = torch.Generator().manual_seed(2)
    m, n, k = 64, 128, 128
    w = torch.randn(n, k, generator=gen).to(BF).cuda()
    dy = torch.randn(m, n, generator=gen).to(BF).cuda()
    x8, c8 = mg.quantise(torch.randn(m, k, generator=gen).cuda()), mg.quantise(torch.randn(m, n, generator=gen).cuda())
    x8[1][5, 2] = 255
    c8[1][9, 1] = 255
    dx, dw, db = mg.linear_backward(dy, x8, w, c=c8, act="gelu", x_dtype="e4m3", c_dtype="e4m3")
    nan = torch.isnan
    assert nan(dx[9]).all() and not nan(dx[:9]).any() and not nan(dx[10:]).any()
    assert nan(db[32:64]).all() and not nan(db[:32]).any() and not nan(db[64:]).any()
    assert nan(dw[:, 64:96]).all() and nan(dw[32:64]).all()
    rest = dw.clone()
    rest[:, 64:96] = 0
    rest[32:64] = 0
    assert not nan(rest).any()


def test_no_rows_backward():
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, 64, dtype=BF, device="cuda")
    p = mg.quantise(e)
    dx, dw, db = mg.linear_backward(e, p, w, c=p, act="gelu", x_dtype="e4m3", c_dtype="e4m3")
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    y, (c, s) = mg.linear(e, w, act="gelu", save_c="e4m3")
    assert y.shape == (0, 64) and c.shape == (0, 64) and s.shape == (0, 2)


def test_other_stream_and_graph():
    gen = torch.Generator().manual_seed(2)
    m, n, k = 555, 512, 384
    x, w = torch.randn(m, k, generator=gen).to(BF).cuda(), (torch.randn(n, k, generator=gen) / 20).to(BF).cuda()
    dy = torch.randn(m, n // 2, generator=gen).to(BF).cuda()

    def step(stream=None):
        x8 = mg.quantise(x, sf_layout="kplanes", stream=stream)
        y, c8 = mg.linear(x, w, act="swiglu", save_c="e4m3", stream=stream)
        return (y, *mg.linear_backward(dy, x8, w, c=c8, act="swiglu", x_dtype="e4m3", c_dtype="e4m3", sf_layout="kplanes",
                                       stream=stream), mg.dequantise(x8, sf_layout="kplanes", stream=stream))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.randn(100000, device="cuda").sum().item()
