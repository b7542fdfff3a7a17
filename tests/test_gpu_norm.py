"""GPU tests of rms_norm and its gradient against the float64 reference."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import more_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = {BF: ref.BF16, F32: ref.F32}


def make(t, h, x_kind, kind, residual, seed=1, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    channel = torch.exp(torch.randn(1, h, generator=gen))
    x = (torch.randn(t, h, generator=gen) * channel * scale).to(x_kind)
    r = (torch.randn(t, h, generator=gen) * 3 * scale).to(kind) if residual else None
    return x, r, torch.rand(h, generator=gen) + 0.5, gen


def cuda(t):
    return None if t is None else t.cuda()


def check_forward(t, h, x_kind=BF, kind=BF, residual=True, dtype="bf16", copy=None, layout="row_major", seed=1, eps=1e-6):
    x, r, w, _ = make(t, h, x_kind, kind, residual, seed)
    print(f"[gpu-case] rms_norm {t}x{h} x={x_kind} stream={kind} residual={residual} {dtype} copy={copy} {layout}", flush=True)
    got = mg.rms_norm(x.cuda(), w.cuda(), residual=cuda(r), eps=eps, dtype=dtype, copy=copy, sf_layout=layout)
    parts = [got] if not residual and copy is None else list(got)
    stored = x
    if residual:
        stored = parts.pop().cpu()
        exact = x.double() + r.double()
        assert stored.dtype is kind
        # x + r in fp32, then rounded to the stream's type
        assert ((stored.double() - exact).abs() <= (EPS[kind] + ref.F32) * exact.abs() * 1.01).all()
    want = ref.rms_norm(stored, w, eps)
    if dtype == "bf16":
        y = parts.pop(0).cpu()
        assert y.dtype is BF and ((y.double() - want).abs() <= (ref.BF16 + ref.Y_OFF) * want.abs() * 1.01 + 1e-38).all()
    fmt = copy if dtype == "bf16" else dtype
    if fmt:
        codes, sf = parts.pop(0)
        ref.check_mx(codes, ref.rowmajor(sf.cpu(), layout), fmt, want, ref.Y_OFF * want.abs())
    assert not parts


@pytest.mark.parametrize("t,h", [(1, 8), (1, 2048), (2, 16), (3, 520), (5, 2048), (7, 1000), (33, 512), (64, 4096),
                                 (130, 1408), (17, 8192), (3, 16384), (2, 32768), (1, 32760), (1001, 2056)])
@pytest.mark.parametrize("x_kind,kind,residual", [(BF, BF, True), (BF, F32, True), (F32, F32, True), (BF, BF, False),
                                                  (F32, F32, False)])
def test_forward(t, h, x_kind, kind, residual):
    check_forward(t, h, x_kind, kind, residual, seed=t + h)


@pytest.mark.parametrize("dtype", ["e4m3", "e5m2", "e2m1x2"])
@pytest.mark.parametrize("layout", ["row_major", "kplanes"])
@pytest.mark.parametrize("t,h", [(1, 256), (5, 2048), (33, 768), (130, 4096), (3, 32768), (257, 2304)])
def test_forward_mx(t, h, dtype, layout):
    check_forward(t, h, dtype=dtype, layout=layout, seed=t)
    check_forward(t, h, F32, F32, False, dtype=dtype, layout=layout, seed=t + 1)
    check_forward(t, h, BF, F32, True, copy=dtype, layout=layout, seed=t + 2)
    check_forward(t, h, BF, BF, False, copy=dtype, layout=layout, seed=t + 3)


@pytest.mark.parametrize("h", [128, 384, 1152])
def test_forward_mx_odd_widths(h):
    for dtype in ("e4m3", "e5m2"):
        check_forward(9, h, dtype=dtype, layout="kplanes")


@pytest.mark.parametrize("h", [8, 16, 24, 56, 64, 72, 120, 128, 136, 248, 256, 264, 504])
@pytest.mark.parametrize("t", [1, 7, 33, 301, 4099])
@pytest.mark.parametrize("kind", [BF, F32])
def test_narrow_rows(t, h, kind):
    """Several rows a wave."""
    check_forward(t, h, BF, kind, True, seed=t + h)
    check_backward(t, h, kind, seed=t + h)
    if h % 128 == 0:
        for layout in ("row_major", "kplanes"):
            check_forward(t, h, BF, kind, True, dtype="e4m3", layout=layout, seed=t)
            check_forward(t, h, BF, kind, True, copy="e5m2", layout=layout, seed=t)
    if h % 256 == 0:
        check_forward(t, h, kind, kind, False, dtype="e2m1x2", layout="kplanes", seed=t)


def test_the_copy_is_the_output():
    """The MX copy beside a BF16 y, the MX y alone, and both y's: the same numbers."""
    x, r, w, _ = make(77, 1024, BF, BF, True)
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    y, (c, s), h = mg.rms_norm(x, w, residual=r, copy="e4m3")
    (c2, s2), h2 = mg.rms_norm(x, w, residual=r, dtype="e4m3")
    y2, h3 = mg.rms_norm(x, w, residual=r)
    assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(h, h3)
    assert torch.equal(mg.rms_norm(h, w), y)            # the norm is the one of the stored sum


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("scale", [1e-30, 1e-15, 1e15, 1e30, 1e37])
def test_sums_neither_overflow_nor_vanish(kind, scale):
    x, _, w, gen = make(9, 1408, kind, kind, False, scale=1.0)
    x = (x.double().clamp(-8, 8) * scale).to(kind)
    for eps in (1e-6, 1e-40):
        y = mg.rms_norm(x.cuda(), w.cuda(), eps=eps).cpu().double()
        want = ref.rms_norm(x, w, torch.tensor(eps, dtype=F32).double())
        assert torch.isfinite(y).all()
        assert ((y - want).abs() <= (ref.BF16 + ref.Y_OFF) * want.abs() * 1.01 + 2.0 ** -134).all(), (kind, scale, eps)
    dy = torch.randn(9, 1408, generator=gen).to(BF)
    for eps in (1e-6, 1e-40):
        e = torch.tensor(eps, dtype=F32).double()
        dx, dw = mg.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=eps)
        want, bound, wdw, bdw = ref.rms_norm_backward(dy, x, w, e)
        most = torch.finfo(kind).max
        ok = want.abs() < most / 2                     # (gradients of a vanishing row may leave the type's range)
        assert ((dx.cpu().double() - want).abs() <= bound + EPS[kind] * want.abs() + 2.0 ** -126)[ok].all(), (scale, eps)
        assert ((dw.cpu().double() - wdw).abs() <= bdw + 1e-38).all()


def test_rows_of_zeros_and_not_numbers():
    x = torch.zeros(6, 512, dtype=BF)
    x[1, 5], x[2, 7], x[3] = math.nan, math.inf, 1.0
    w = torch.full((512,), 2.0)
    y = mg.rms_norm(x.cuda(), w.cuda()).cpu().float()
    assert (y[0] == 0).all() and (y[4:] == 0).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 7]) and (y[2, :7] == 0).all() and (y[2, 8:] == 0).all()      # inf / inf, finite / inf
    assert (y[3] == 2.0).all()
    (codes, sf) = mg.rms_norm(x.cuda(), w.cuda(), dtype="e4m3")
    assert (sf[1] == 255).all() and (codes[1] == 0).all() and (sf[0] == 0).all() and (sf[2, 0] == 255) and (sf[2, 1:] == 0).all()
    dy = torch.ones(6, 512, dtype=BF)
    dx, _ = mg.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), need=("dx",))
    assert torch.isnan(dx[1]).all() and not torch.isnan(dx[[0, 3, 4, 5]]).any()


def check_backward(t, h, kind, dh=True, seed=1, need=("dx", "dw")):
    x, _, w, gen = make(t, h, kind, kind, False, seed)
    dy = torch.randn(t, h, generator=gen).to(BF)
    g = torch.randn(t, h, generator=gen).to(kind) if dh else None
    print(f"[gpu-case] rms_norm backward {t}x{h} {kind} dh={dh} {need}", flush=True)
    dx, dw = mg.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), dh=cuda(g), need=need)
    want, bound, wdw, bdw = ref.rms_norm_backward(dy, x, w, 1e-6, g)
    assert (dx is None) == ("dx" not in need) and (dw is None) == ("dw" not in need)
    if dx is not None:
        assert dx.dtype is kind
        bad = (dx.cpu().double() - want).abs() > bound + EPS[kind] * want.abs() * 1.01
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    if dw is not None:
        assert ((dw.cpu().double() - wdw).abs() <= bdw + 1e-30).all()
    return dx, dw


@pytest.mark.parametrize("t,h", [(1, 8), (1, 2048), (3, 520), (7, 1000), (33, 512), (64, 4096), (130, 1408), (17, 8192),
                                 (3, 16384), (2, 32768), (1001, 2056), (5000, 256), (2049, 2048)])
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("dh", [True, False])
def test_backward(t, h, kind, dh):
    check_backward(t, h, kind, dh, seed=t + h)


def test_backward_parts():
    a = check_backward(300, 1024, BF)
    b = check_backward(300, 1024, BF, need=("dx",))
    c = check_backward(300, 1024, BF, need=("dw",))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], c[1])


def test_in_place():
    """The sum in the residual's place, and dx in dh's through the C function."""
    x, r, w, gen = make(50, 520, BF, F32, True)
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    y, h = mg.rms_norm(x, w, residual=r)
    r2 = r.clone()
    y2, h2 = mg.rms_norm(x, w, residual=r2, h=r2)
    assert h2 is r2 and torch.equal(h, h2) and torch.equal(y, y2)
    dy, dh = torch.randn(50, 520, generator=gen).to(BF).cuda(), torch.randn(50, 520, generator=gen).cuda()
    dx, _ = mg.rms_norm_backward(dy, h, w, dh=dh, need=("dx",))
    p = mg.moegg_norm_problem(50, 520, 5, 5, 0, 0, 1e-6)
    a = mg.moegg_norm_args(weight=w.data_ptr(), h=h.data_ptr(), dy=dy.data_ptr(), dh=dh.data_ptr(), dx=dh.data_ptr())
    assert mg._load().moegg_rms_norm_backward(p, a, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dh, dx)


def test_vectors_at_any_multiple_of_4_bytes():
    x, r, w, gen = make(40, 1032, BF, BF, True)
    wide = torch.zeros(1032 + 5, device="cuda")
    want = mg.rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
    dy = torch.randn(40, 1032, generator=gen).to(BF).cuda()
    grads = mg.rms_norm_backward(dy, want[1], w.cuda())
    for shift in (1, 2, 3):
        view = wide[shift:shift + 1032]
        view.copy_(w)
        got = mg.rms_norm(x.cuda(), view, residual=r.cuda())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g = mg.rms_norm_backward(dy, want[1], view)
        assert torch.equal(g[0], grads[0]) and torch.equal(g[1], grads[1])
    with pytest.raises(mg.MoeggError, match="aligned"):
        mg.rms_norm(torch.zeros(9 * 1032 + 4, dtype=BF, device="cuda")[4:].view(9, 1032), w.cuda())


def test_no_rows():
    w = torch.ones(256, device="cuda")
    e = torch.empty(0, 256, dtype=BF, device="cuda")
    y, (c, s), h = mg.rms_norm(e, w, residual=e, copy="e4m3")
    assert y.shape == (0, 256) and c.shape == (0, 256) and s.shape == (0, 8) and h.shape == (0, 256)
    dx, dw = mg.rms_norm_backward(e, e, w)
    assert dx.shape == (0, 256) and (dw == 0).all()
    dx, dw = mg.rms_norm_backward(e, e, w, need=("dx",))
    assert dx.shape == (0, 256) and dw is None


def test_many_rows():
    """More elements than 32 bits count."""
    t, h = (1 << 20) + 3, 4096
    x = torch.zeros(t, h, dtype=BF, device="cuda")
    x[-1] = torch.arange(h, device="cuda").remainder(7).to(BF)
    w = torch.ones(h, device="cuda")
    y, r = mg.rms_norm(x, w, residual=x, h=None)
    assert (r[-1] == 2 * x[-1]).all()
    want = ref.rms_norm(r[-1:].cpu(), w.cpu(), 1e-6)
    assert ((y[-1:].cpu().double() - want).abs() <= (ref.BF16 + ref.Y_OFF) * 1.01 * want.abs()).all()
    del y, r
    codes, sf = mg.rms_norm(x, w, dtype="e4m3", sf_layout="kplanes")
    want = ref.rms_norm(x[-1:].cpu(), w.cpu(), 1e-6)
    ref.check_mx(codes[-1:], sf[:, -1].reshape(1, -1), "e4m3", want, ref.Y_OFF * want.abs())
    del codes, sf
    dx, dw = mg.rms_norm_backward(x, x, w)
    want, bound, wdw, bdw = ref.rms_norm_backward(x[-1:].cpu(), x[-1:].cpu(), w.cpu(), 1e-6)
    assert ((dx[-1:].cpu().double() - want).abs() <= bound + ref.BF16 * 1.01 * want.abs()).all()
    assert ((dw.cpu().double() - wdw).abs() <= bdw).all()


def test_other_stream_and_graph():
    x, r, w, gen = make(333, 2048, BF, BF, True)
    dy = torch.randn(333, 2048, generator=gen).to(BF).cuda()
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    want = mg.rms_norm(x, w, residual=r, copy="e5m2")
    grads = mg.rms_norm_backward(dy, want[-1], w, dh=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mg.rms_norm(x, w, residual=r, copy="e5m2", stream=side)
    g2 = mg.rms_norm_backward(dy, got[-1], w, dh=r, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = mg.rms_norm(x, w, residual=r, copy="e5m2")
        g3 = mg.rms_norm_backward(dy, cap[-1], w, dh=r)
    for _ in range(3):
        for t in (cap[0], cap[1][0], cap[1][1], cap[2], *g3):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((got, g2), (cap, g3)):
            assert torch.equal(a[0], want[0]) and torch.equal(a[1][0], want[1][0]) and torch.equal(a[1][1], want[1][1])
            assert torch.equal(a[2], want[2]) and torch.equal(b[0], grads[0]) and torch.equal(b[1], grads[1])
        torch.randn(100000, device="cuda").sum().item()
