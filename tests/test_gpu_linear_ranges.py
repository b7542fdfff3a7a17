"""linear and its gradients over the whole range of BF16 numbers, past 2^31
elements, and bit for bit from call to call."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

F32_MAX, BF16_MAX = torch.finfo(torch.float32).max, torch.finfo(torch.bfloat16).max


def every_bf16(seed):
    """(1020, 64): every finite BF16 number once, shuffled."""
    bits = torch.arange(0x7F80, dtype=torch.int32)
    v = torch.cat([bits, bits | 0x8000]).to(torch.int16).view(torch.bfloat16)
    return v[torch.randperm(v.numel(), generator=torch.Generator().manual_seed(seed))].reshape(-1, 64)


def agree(got, want, bound, most):
    """Within the bound; an infinity where the number is too large for the type."""
    got = got.cpu().double()
    assert not torch.isnan(got).any()
    over, fine = want.abs() > most * 1.005, want.abs() < most * 0.995      # (between them a rounding decides)
    assert torch.equal(got[over], torch.sign(want[over]) * math.inf)
    bad = ((got - want).abs() > bound) & fine
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [slice(0, 12), slice(0, None)])
@pytest.mark.parametrize("act", ["none", "swiglu", "srelu", "gelu"])
def test_every_pre_activation(act, rows, dtype):
    """w is the identity: z is x itself, exactly, and y the activation of every number."""
    for seed in range(3):
        x = every_bf16(seed)[rows].contiguous()
        print(f"[gpu-case] linear every bf16 {act} rows={x.shape[0]} {dtype}", flush=True)
        y, c = mg.linear(x.cuda(), torch.eye(64, dtype=torch.bfloat16, device="cuda"), act=act, save_c=True, dtype=dtype)
        assert torch.equal(c.cpu().float(), x.float())
        z, eps = x.double(), ref.BF16 if dtype == "bf16" else ref.F32
        agree(y, ref.act(z, act), ref.linear_bound(z, torch.zeros_like(z), 64, act, None, eps),
              BF16_MAX if dtype == "bf16" else F32_MAX)


@pytest.mark.parametrize("rows", [slice(0, 12), slice(0, None)])
@pytest.mark.parametrize("act", ["swiglu", "srelu", "gelu"])
def test_every_saved_pre_activation(act, rows):
    """w is the identity: dx is dz, for every c."""
    for seed in range(3):
        c = every_bf16(seed + 10)[rows].contiguous()
        m, n_out = c.shape[0], 32 if act == "swiglu" else 64
        dy = torch.randn(m, n_out, generator=torch.Generator().manual_seed(seed)).clamp(-2, 2).to(torch.bfloat16)
        print(f"[gpu-case] linear backward every bf16 {act} rows={m}", flush=True)
        eye = torch.eye(64, dtype=torch.bfloat16, device="cuda")
        dx, _, _ = mg.linear_backward(dy.cuda(), torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda"), eye, c=c.cuda(), act=act,
                                      need=("dx",))
        d, z = dy.double(), c.double()
        if act == "swiglu":
            v, e = z.reshape(m, 1, 2, 32), d.reshape(m, 1, 32)
            s = torch.sigmoid(v[:, :, 1])
            dz = torch.stack([e * v[:, :, 1] * s, e * v[:, :, 0] * (s + v[:, :, 1] * s * torch.sigmoid(-v[:, :, 1]))], 2).reshape(m, 64)
            # the factor s (1 + g (1 - s)) is off by 24 roundings of numbers up to 1.3, and so, times x, is the gate's half;
            # g s by 8 of g's
            off = torch.stack([e.abs() * v[:, :, 1].abs() * 8 * ref.F32, e.abs() * v[:, :, 0].abs() * 32 * ref.F32], 2).reshape(m, 64)
        elif act == "srelu":
            dz, off = d * 2.0 * z.clamp(min=0.0), 0.0
        else:
            s = torch.sigmoid(2.0 * ref.C * (z + ref.A * z ** 3))
            dz = d * (s + z * s * torch.sigmoid(-2.0 * ref.C * (z + ref.A * z ** 3)) * 2.0 * ref.C * (1 + 3 * ref.A * z * z))
            off = d.abs() * 64 * ref.F32
        # dz rounds to an infinity past bf16's range; times the identity's zeros that is NaN in the row's other columns
        # (and in its own where there is another one): only rows without such a number are compared with dz, and what
        # the others hold is their sum's
        over, between = dz.abs() > BF16_MAX * 1.005, (dz.abs() > BF16_MAX * 0.995).logical_and(dz.abs() < BF16_MAX * 1.005)
        fine = ~(over | between).any(1)
        off = off if isinstance(off, float) else off[fine]
        agree(dx.cpu()[fine], dz[fine], off + (ref.BF16 + 16 * ref.F32) * dz[fine].abs() + 1e-38, BF16_MAX)
        sure = over.any(1) & ~between.any(1)
        alone = over & (over.sum(1, keepdim=True) == 1)
        want = torch.where(alone, torch.sign(dz) * math.inf, math.nan)
        assert torch.equal(torch.isnan(dx.cpu()[sure]), torch.isnan(want[sure]))
        assert torch.equal(dx.cpu().double()[sure][alone[sure]], want[sure][alone[sure]])


@pytest.mark.parametrize("act,dtype,m", [("srelu", "bf16", 1100000), ("gelu", "f32", 1099909), ("none", "f32", 1100000),
                                         ("swiglu", "bf16", 2200000), ("swiglu", "f32", 2199818)])
def test_results_past_two_to_the_31_elements(act, dtype, m):
    """y, c and the residual: the first and the last rows (also where few rows follow whole tiles)."""
    n, k = 2048, 64
    n_out = n // 2 if act == "swiglu" else n
    assert m * n_out > 2 ** 31
    print(f"[gpu-case] linear m={m} n={n} k={k} {act} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(m, k, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    b = torch.randn(n, generator=gen, device="cuda")
    res = torch.randn(m, n_out, generator=gen, device="cuda", dtype=torch.bfloat16)
    y, c = mg.linear(x, w, bias=b, act=act, residual=res, save_c=True, dtype=dtype)
    half = (2 ** 31 // n_out) // 128 * 128                 # where y's element numbers pass 32 bits
    for part in (slice(0, 200), slice(half - 100, half + 300), slice(m - 200, m)):
        xd = x[part].double()
        z = xd @ w.double().t() + b.double()
        mag = xd.abs() @ w.double().abs().t() + b.double().abs()
        assert ((c[part].double() - z).abs() <= (k + 8) * ref.F32 * mag * 1.01 + ref.BF16 * z.abs()).all()
        want = ref.act(z, act) + res[part].double()
        bound = ref.linear_bound(z, mag, k, act, res[part], ref.BF16 if dtype == "bf16" else ref.F32)
        assert ((y[part].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_gradients_past_two_to_the_31_elements(act):
    """dz in the workspace: dx of the first and last rows, db, and a corner of dw."""
    m, n, k = 1100000, 2048, 64
    n_out = n // 2 if act == "swiglu" else n
    print(f"[gpu-case] linear backward m={m} n={n} k={k} {act}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(m, k, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    c = torch.randn(m, n, generator=gen, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(m, n_out, generator=gen, device="cuda", dtype=torch.bfloat16)
    dx, dw, db = mg.linear_backward(dy, x, w, c=c, act=act, dw_dtype="f32")
    for part in (slice(0, 200), slice(2 ** 31 // n - 100, 2 ** 31 // n + 100), slice(m - 200, m)):
        r, bound = ref.linear_backward(dy[part].cpu(), x[part].cpu(), w.cpu(), c[part].cpu(), act)["dx"]
        assert ((dx[part].cpu().double() - r).abs() <= bound * (1 + ref.BF16) + ref.BF16 * r.abs()).all()
    # column 0 (and its pair's gate 32): db and a corner of dw over all rows
    cols = [0, 32] if act == "swiglu" else [0]
    r = torch.zeros(len(cols), k, dtype=torch.float64, device="cuda")
    mag, s, sa = r.clone(), torch.zeros(len(cols), dtype=torch.float64, device="cuda"), torch.zeros(len(cols), dtype=torch.float64, device="cuda")
    for at in range(0, m, 100000):
        part = slice(at, at + 100000)
        d, z, xd = dy[part, 0].double(), c[part].double(), x[part].double()
        if act == "swiglu":
            sg = torch.sigmoid(z[:, 32])
            dz = torch.stack([d * z[:, 32] * sg, d * z[:, 0] * sg * (1 + z[:, 32] * (1 - sg))], 1)
            ev = torch.stack([d.abs()] * 2, 1) * torch.maximum(z[:, 0].abs(), z[:, 32].abs())[:, None] * 32 * ref.F32
        else:
            sg = torch.sigmoid(2 * ref.C * (z[:, 0] + ref.A * z[:, 0] ** 3))
            dz = (d * (sg + z[:, 0] * sg * (1 - sg) * 2 * ref.C * (1 + 3 * ref.A * z[:, 0] ** 2)))[:, None]
            ev = d.abs()[:, None] * 64 * ref.F32
        ev = ev + 16 * ref.F32 * dz.abs()
        r += dz.t() @ xd
        mag += (ev + (ref.BF16 + (m + 8) * ref.F32) * dz.abs()).t() @ xd.abs()
        s += dz.sum(0)
        sa += (ev + (m + 8) * ref.F32 * dz.abs()).sum(0)
    assert ((dw[cols].double() - r).abs() <= mag * (1 + ref.F32) + ref.F32 * r.abs()).all()
    assert ((db[cols].double() - s).abs() <= sa * (1 + ref.F32)).all()


def poison(seed):
    """What the allocator hands out next holds no zeros: NaN, infinities, large numbers."""
    held = [torch.full((1 << i,), (0xFF, 0x7F, 0x5A)[seed % 3], dtype=torch.uint8, device="cuda") for i in range(9, 30)]
    del held


@pytest.mark.parametrize("act", ["none", "swiglu", "gelu"])
@pytest.mark.parametrize("m,n,k,groups", [(5, 320, 200, 0), (300, 256, 4096, 0), (4099, 2048, 200, 0), (16384, 2816, 2048, 0),
                                          (96, 192, 264, 64), (2000, 512, 328, 3), (24571, 2048, 1408, 64)])
def test_the_same_bits_in_every_call(m, n, k, groups, act):
    """Forward and backward five times, on memory that held other things each time."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(*((groups, n, k) if groups else (n, k)), generator=gen, device="cuda") / math.sqrt(k)).to(torch.bfloat16)
    b = torch.randn(*((groups, n) if groups else (n,)), generator=gen, device="cuda")
    dy = torch.randn(m, n // 2 if act == "swiglu" else n, generator=gen, device="cuda").to(torch.bfloat16)
    off = None
    if groups:
        off = torch.sort(torch.randint(0, m, (groups,), generator=gen, device="cuda", dtype=torch.int32)).values
        off[-1] = m
    print(f"[gpu-case] linear repeated m={m} n={n} k={k} {act} groups={groups}", flush=True)

    def step():
        y, c = mg.linear(x, w, bias=b, act=act, offsets=off, save_c=True)
        return (y, c, *mg.linear_backward(dy, x, w, c=None if act == "none" else c, act=act, offsets=off, dw_dtype="f32"))
    first = step()
    for rep in range(4):
        poison(rep)
        for u, v in zip(first, step()):
            assert torch.equal(u, v)
