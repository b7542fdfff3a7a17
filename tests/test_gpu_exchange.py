"""GPU tests of the token exchange: sort, dispatch, combine and their gradients."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def make_ids(t, k, e, seed, drop=0.1, skew=False):
    gen = torch.Generator().manual_seed(seed)
    if skew:
        ids = (torch.rand(t, k, generator=gen) ** 6 * e).long().clamp(max=e - 1)
    else:
        ids = torch.randint(0, e, (t, k), generator=gen)
    ids[torch.rand(t, k, generator=gen) < drop] = -1
    return ids.to(torch.int32), gen


def check_plan(ids, e, ma, weights=None):
    t, k = ids.shape
    print(f"[gpu-case] sort {t}x{k} experts={e} m_aligned={ma}", flush=True)
    plan = mg.sort_tokens(ids.cuda(), e, m_aligned=ma, weights=None if weights is None else weights.cuda())
    off, row_of, slot_of = ref.sort(ids, e, ma, plan.rows)
    assert plan.rows == mg.sort_rows(t, k, e, ma) and plan.rows >= int(off[-1])
    assert torch.equal(plan.padded_offsets.cpu().long(), off)
    assert torch.equal(plan.row_of.cpu().long(), row_of)
    assert torch.equal(plan.slot_of.cpu().long(), slot_of)
    if weights is not None:
        want = torch.where(slot_of >= 0, weights.reshape(-1)[slot_of.clamp(min=0)] if slot_of.numel() and t else 0.0, 0.0)
        assert torch.equal(plan.prob.cpu(), want.float())
    return plan, off, row_of, slot_of


@pytest.mark.parametrize("t,k,e,ma", [
    (1, 1, 1, 1), (1, 6, 64, 128), (3, 6, 64, 1), (7, 2, 5, 3), (100, 8, 8, 16), (341, 6, 64, 128), (257, 8, 128, 32),
    (700, 3, 1000, 128), (1000, 6, 64, 128), (4099, 4, 1024, 1), (16384, 6, 64, 128), (5000, 32, 3, 65536),
])
@pytest.mark.parametrize("skew", [False, True])
def test_sort(t, k, e, ma, skew):
    ids, gen = make_ids(t, k, e, seed=t + e, skew=skew)
    check_plan(ids, e, ma, torch.rand(t, k, generator=gen))
    check_plan(ids, e, ma)


def test_sort_one_expert_takes_all_and_none():
    ids = torch.full((3000, 2), 5, dtype=torch.int32)
    check_plan(ids, 9, 128)
    check_plan(torch.full((3000, 2), -1, dtype=torch.int32), 9, 128, torch.rand(3000, 2))
    # numbers that are no expert drop the slot
    check_plan(torch.tensor([[9, 0], [2 ** 31 - 1, -2 ** 31], [8, -7]], dtype=torch.int32), 9, 4)


def test_sort_many_slots():
    """More slots than 256 blocks of the smallest chunk: longer chunks."""
    ids, gen = make_ids(200003, 3, 100, seed=8, skew=True)
    check_plan(ids, 100, 128, torch.rand(200003, 3, generator=gen))


def test_sort_empty():
    plan, off, _, _ = check_plan(torch.empty(0, 4, dtype=torch.int32), 6, 128)
    assert plan.rows == 0 and off.tolist() == [0] * 6


def test_sort_into_more_rows_than_needed():
    """Rows behind the last expert belong to no slot, up to the size the caller chose."""
    import ctypes
    ids, gen = make_ids(50, 2, 7, seed=2)
    w = torch.rand(50, 2, generator=gen)
    rows = mg.sort_rows(50, 2, 7, 16) + 1000
    off, row_of, slot_of = ref.sort(ids, 7, 16, rows)
    o = [torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (7, 100, rows)]
    prob = torch.full((rows,), 7.0, device="cuda")
    p = mg.moegg_sort_problem(num_tokens=50, top_k=2, num_experts=7, m_aligned=16, rows=rows)
    d_ids, d_w = ids.cuda(), w.cuda()
    st = mg._load().moegg_sort(ctypes.byref(p), d_ids.data_ptr(), d_w.data_ptr(), o[0].data_ptr(), o[1].data_ptr(),
                               o[2].data_ptr(), prob.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(o[0].cpu().long(), off) and torch.equal(o[1].cpu().long(), row_of.reshape(-1))
    assert torch.equal(o[2].cpu().long(), slot_of) and (prob.cpu()[slot_of < 0] == 0).all()


MARK = 0x5A


def filled(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(MARK)
    return t


def decode_equal(a, b, sign):
    """Codes equal, a negative zero counting as zero."""
    def plain(c):
        return np.where((c & ~np.uint8(sign)) == 0, 0, c)
    return np.array_equal(plain(a), plain(b))


def nibbles(c):
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)


def same_codes(got, want, fmt):
    if fmt == "e2m1x2":
        return decode_equal(nibbles(got), nibbles(want), 8)
    return decode_equal(got, want, 0x80)


def rowmajor(sf, layout):
    return sf if layout == "row_major" else sf.transpose(1, 0, 2).reshape(sf.shape[1], -1)


@pytest.mark.parametrize("t,k,e,ma,h", [(1, 1, 1, 1, 8), (5, 2, 4, 1, 264), (33, 6, 16, 32, 512), (130, 3, 7, 128, 1288),
                                        (1, 6, 64, 128, 2048), (77, 32, 40, 8, 640), (600, 4, 8, 128, 4096)])
def test_dispatch_and_combine(t, k, e, ma, h):
    ids, gen = make_ids(t, k, e, seed=t + h)
    x = torch.randn(t, h, generator=gen).to(torch.bfloat16)
    w, res = torch.rand(t, k, generator=gen), torch.randn(t, h, generator=gen).to(torch.bfloat16)
    plan, off, row_of, slot_of = check_plan(ids, e, ma)
    print(f"[gpu-case] dispatch H={h}", flush=True)
    buf = filled((plan.rows, h), torch.bfloat16)
    a = mg.dispatch(x.cuda(), plan, out=buf)
    assert a is buf
    used = int(off[-1])
    assert torch.equal(a.cpu().double()[:used], ref.dispatch(x, slot_of, k)[:used])
    assert (a[used:].view(torch.uint8) == MARK).all()          # behind the last expert: as it was
    rows = torch.randn(plan.rows, h, generator=gen).to(torch.bfloat16)
    rows[slot_of < 0] = math.nan                               # padding is never read
    for weights in (w, None):
        for residual in (res, None):
            y = mg.combine(rows.cuda(), plan, weights=None if weights is None else weights.cuda(),
                           residual=None if residual is None else residual.cuda())
            r, mag = ref.combine(rows, row_of, weights, residual)
            assert ((y.cpu().double() - r).abs() <= ref.BF16 * r.abs() + (k + 2) * ref.F32 * 2 * mag).all()
    # in place on the residual
    inout = res.cuda()
    y2 = mg.combine(rows.cuda(), plan, weights=w.cuda(), residual=inout, out=inout)
    assert y2 is inout and torch.equal(y2, mg.combine(rows.cuda(), plan, weights=w.cuda(), residual=res.cuda()))
    dx = mg.dispatch_backward(rows.cuda(), plan)
    r, mag = ref.combine(rows, row_of)
    assert ((dx.cpu().double() - r).abs() <= ref.BF16 * r.abs() + (k + 2) * ref.F32 * mag).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1x2"])
@pytest.mark.parametrize("layout", ["row_major", "kplanes"])
@pytest.mark.parametrize("t,k,e,ma,h", [(1, 1, 1, 1, 256), (41, 3, 6, 128, 768), (9, 6, 64, 1, 2048), (300, 2, 4, 128, 1280)])
def test_dispatch_mx(fmt, layout, t, k, e, ma, h):
    ids, gen = make_ids(t, k, e, seed=t + h)
    x = (torch.randn(t, h, generator=gen) * torch.exp(3 * torch.randn(t, 1, generator=gen))).to(torch.bfloat16)
    x[:, 32:64] = 0.0
    x[0, :32] = 448.0 * 2.0 ** -4                              # amax on the border of two scales
    x[-1, 64:96] = 7.5
    plan, off, _, slot_of = check_plan(ids, e, ma)
    shape = (plan.rows, h // 2 if fmt == "e2m1x2" else h)
    sshape = (h // 128, plan.rows, 4) if layout == "kplanes" else (plan.rows, h // 32)
    out = filled(shape, torch.uint8), filled(sshape, torch.uint8)
    codes, sf = mg.dispatch(x.cuda(), plan, dtype=fmt, sf_layout=layout, out=out)
    used = int(off[-1])
    want, byte = ref.mx_encode(ref.dispatch(x, slot_of, k)[:used], fmt)
    got, gsf = codes.cpu().numpy(), rowmajor(sf.cpu().numpy(), layout)
    assert np.array_equal(gsf[:used], byte) and same_codes(got[:used], want, fmt)
    assert (got[used:] == MARK).all() and (gsf[used:] == MARK).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1x2"])
def test_dispatch_mx_special_values(fmt):
    """Subnormals, the largest numbers, infinities and NaN, every bf16 magnitude as a block's amax."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)           # every finite bf16 >= 0
    h = 256
    x = torch.zeros(bits.numel() // 8 + 1, 8, 32, dtype=torch.int32)
    x.reshape(-1, 32)[:bits.numel(), 0] = bits
    x.reshape(-1, 32)[:bits.numel(), 7] = bits // 2 | 0x8000    # and something smaller of the other sign
    x = x.reshape(-1, h).to(torch.int16).view(torch.bfloat16)
    bad = torch.zeros(4, h, dtype=torch.bfloat16)
    bad[0, 3], bad[1, 40], bad[2, 255] = math.inf, math.nan, -math.inf
    bad[:, 100] = 1.0
    x = torch.cat([x, bad])
    t = x.shape[0]
    ids = torch.zeros(t, 1, dtype=torch.int32)
    plan = mg.sort_tokens(ids.cuda(), 1, m_aligned=1)
    codes, sf = mg.dispatch(x.cuda(), plan, dtype=fmt)
    want, byte = ref.mx_encode(x.double(), fmt)
    assert np.array_equal(sf.cpu().numpy(), byte)
    assert same_codes(codes.cpu().numpy(), want, fmt)
    assert (byte[-4:] == 255).sum() == 3


@pytest.mark.parametrize("t,k,e,ma,h", [(1, 1, 1, 1, 8), (5, 2, 4, 1, 264), (33, 6, 16, 32, 512), (130, 3, 7, 128, 1288),
                                        (64, 9, 64, 128, 2048), (20, 32, 40, 8, 640), (600, 4, 8, 128, 4096)])
def test_combine_backward(t, k, e, ma, h):
    ids, gen = make_ids(t, k, e, seed=t + h + 1)
    dy = torch.randn(t, h, generator=gen).to(torch.bfloat16)
    w = torch.rand(t, k, generator=gen)
    plan, off, row_of, slot_of = check_plan(ids, e, ma)
    rows = torch.randn(plan.rows, h, generator=gen).to(torch.bfloat16)
    rows[slot_of < 0] = math.nan
    used = int(off[-1])
    for weights in (w, None):
        buf = filled((plan.rows, h), torch.bfloat16)
        d, dw = mg.combine_backward(dy.cuda(), plan, rows=rows.cuda(),
                                    weights=None if weights is None else weights.cuda(), out=buf)
        slot_w = torch.ones(plan.rows) if weights is None else w.reshape(-1)[slot_of.clamp(min=0)]
        r = ref.dispatch(dy, slot_of, k) * slot_w.double()[:, None]
        assert ((d.cpu().double() - r).abs() <= (ref.BF16 + 2 * ref.F32) * r.abs())[:used].all()
        assert (d[used:].view(torch.uint8) == MARK).all()
        picked = torch.where((row_of >= 0)[:, :, None], rows.double()[row_of.clamp(min=0).long()], 0.0)
        term = picked * dy.double()[:, None, :]
        assert ((dw.cpu().double() - term.sum(2)).abs() <= (h + 8) * ref.F32 * term.abs().sum(2)).all()
        d2, none = mg.combine_backward(dy.cuda(), plan, weights=None if weights is None else weights.cuda())
        assert none is None and torch.equal(d2[:used], d[:used])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1x2"])
@pytest.mark.parametrize("layout", ["row_major", "kplanes"])
def test_combine_backward_mx(fmt, layout):
    """dy times a weight in MX rows.  Weights are powers of two, so that the products are exact."""
    t, k, e, ma, h = 57, 3, 6, 128, 768
    ids, gen = make_ids(t, k, e, seed=3)
    dy = torch.randn(t, h, generator=gen).to(torch.bfloat16)
    w = torch.exp2(torch.randint(-6, 3, (t, k), generator=gen).float()) * torch.where(torch.rand(t, k, generator=gen) < 0.1, 0.0, 1.0)
    plan, off, row_of, slot_of = check_plan(ids, e, ma)
    rows = torch.randn(plan.rows, h, generator=gen).to(torch.bfloat16)
    (codes, sf), dw = mg.combine_backward(dy.cuda(), plan, rows=rows.cuda(), weights=w.cuda(), dtype=fmt, sf_layout=layout)
    used = int(off[-1])
    r = ref.dispatch(dy, slot_of, k) * w.reshape(-1)[slot_of.clamp(min=0)].double()[:, None]
    want, byte = ref.mx_encode(r[:used], fmt)
    assert np.array_equal(rowmajor(sf.cpu().numpy(), layout)[:used], byte)
    assert same_codes(codes.cpu().numpy()[:used], want, fmt)
    picked = torch.where((row_of >= 0)[:, :, None], rows.double()[row_of.clamp(min=0).long()], 0.0)
    term = picked * dy.double()[:, None, :]
    assert ((dw.cpu().double() - term.sum(2)).abs() <= (h + 8) * ref.F32 * term.abs().sum(2)).all()


def test_unsort():
    ids, gen = make_ids(201, 5, 12, seed=6)
    plan, _, row_of, _ = check_plan(ids, 12, 16)
    v = torch.randn(plan.rows, generator=gen)
    got = mg.unsort(v.cuda(), plan).cpu()
    assert torch.equal(got, torch.where(row_of >= 0, v[row_of.clamp(min=0).long()], 0.0))


def test_foreign_plans_are_not_followed():
    """Rows out of range in a plan count as dropped slots; offsets past the rows end at them."""
    t, k, e, h = 6, 2, 3, 64
    gen = torch.Generator().manual_seed(1)
    row_of = torch.tensor([[0, 50], [-5, 2], [2 ** 31 - 1, 1], [3, -2 ** 31], [4, 5], [10, 9]], dtype=torch.int32)
    slot_of = torch.full((10,), -1, dtype=torch.int32)
    for s, r in enumerate(row_of.reshape(-1).tolist()):
        if 0 <= r < 10:
            slot_of[r] = s
    plan = mg.SortPlan(e, 1, torch.tensor([3, 1000, 2 ** 31 - 1], dtype=torch.int32).cuda(), row_of.cuda(), slot_of.cuda())
    ok = torch.where((row_of >= 0) & (row_of < 10), row_of, -1).long()
    x = torch.randn(t, h, generator=gen).to(torch.bfloat16)
    a = mg.dispatch(x.cuda(), plan).cpu()
    want = torch.zeros(10, h, dtype=torch.bfloat16)
    for s, r in enumerate(ok.reshape(-1).tolist()):
        if r >= 0:
            want[r] = x[s // k]
    assert torch.equal(a, want)
    rows = torch.randn(10, h, generator=gen).to(torch.bfloat16)
    r, _ = ref.combine(rows, ok)
    assert (mg.combine(rows.cuda(), plan).cpu().double() - r).abs().max() < 0.05
    d, dw = mg.combine_backward(x.cuda(), plan, rows=rows.cuda())
    assert torch.equal(d.cpu(), want) and (dw.cpu()[ok < 0] == 0).all()


def test_combine_backward_without_rows():
    """No rows: every slot is a dropped one, whose weight has the gradient 0."""
    t, k, h = 5, 2, 64
    gen = torch.Generator().manual_seed(2)
    dy = torch.randn(t, h, generator=gen).to(torch.bfloat16).cuda()
    plan = mg.SortPlan(3, 1, torch.zeros(3, dtype=torch.int32).cuda(), torch.full((t, k), -1, dtype=torch.int32).cuda(),
                       torch.empty(0, dtype=torch.int32).cuda())
    rows = torch.empty(0, h, dtype=torch.bfloat16).cuda()
    before = torch.full((t, k), 7.0, device="cuda")      # what the next allocation of this size may hold
    del before
    d, dw = mg.combine_backward(dy, plan, rows=rows)
    assert d.shape == (0, h) and (dw == 0).all()
    assert (mg.combine(rows, plan) == 0).all()


def test_more_than_two_to_the_31_elements():
    """Rows whose element numbers pass 32 bits: checked on the last rows."""
    t, k, e, h = 66000, 8, 16, 4096
    print(f"[gpu-case] exchange {t}x{k} H={h}: {t * k * h} elements", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, e, (t, k), generator=gen, device="cuda", dtype=torch.int32)
    plan = mg.sort_tokens(ids, e, m_aligned=1)
    x = torch.randn(t, h, generator=gen, device="cuda").to(torch.bfloat16)
    a = mg.dispatch(x, plan)
    assert a.numel() > 2 ** 31
    token = (plan.slot_of // k).long()
    for part in (slice(0, 500), slice(t * k - 500, t * k)):
        assert torch.equal(a[part], x[token[part]])
    y = mg.combine(a, plan)
    want = (k * x[-300:].float())
    assert ((y[-300:].float() - want).abs() <= 2.0 ** -8 * want.abs()).all()
    d, dw = mg.combine_backward(x, plan, rows=a)
    assert torch.equal(d[-500:], x[token[-500:]])
    sq = (x[-300:].float() ** 2).sum(1, keepdim=True)
    assert ((dw[-300:] - sq).abs() <= h * 2.0 ** -24 * sq).all()
