"""GPU tests of rms_norm and its gradient at the ends of the types' ranges:
rows of the largest numbers, of the smallest, and of both."""
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import more_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: ref.BF16, F32: ref.F32}
# half of the smallest step: what a rounding below the normal numbers is off by at most
LOW = {BF: 2.0 ** -134, F32: 2.0 ** -150}


def rows(h, kind, gen):
    most, least = torch.finfo(kind).max, 2.0 ** (-133 if kind is BF else -149)
    sign = torch.randint(0, 2, (6, h), generator=gen).double() * 2 - 1
    x = torch.empty(6, h, dtype=torch.float64)
    x[0], x[1], x[2] = most, least, 0.0
    x[3] = torch.randn(h, generator=gen).double().clamp(-4, 4) * 1e-38
    x[4] = torch.randn(h, generator=gen).double().clamp(-4, 4)
    x[4, h // 2] = most                                     # one number that all others vanish beside
    x[5] = torch.exp(torch.empty(h).uniform_(-80, 80, generator=gen)).double()
    return (x * sign).to(kind)


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("h", [8, 64, 520, 1408, 8192, 32768])
@pytest.mark.parametrize("eps", [1e-6, 1.5e-45, 3e38])
def test_ends_of_the_range(h, kind, eps):
    gen = torch.Generator().manual_seed(h)
    x = rows(h, kind, gen)
    w = torch.rand(h, generator=gen) + 0.5
    e = torch.tensor(eps, dtype=F32).double()
    print(f"[gpu-case] rms_norm ends of the range {h} {kind} eps={eps}", flush=True)
    y = mg.rms_norm(x.cuda(), w.cuda(), eps=eps).cpu().double()
    want = ref.rms_norm(x, w, e)
    # (h r below the normal numbers is rounded to fp32's lowest step, twice with the weight)
    assert ((y - want).abs() <= (ref.BF16 + ref.Y_OFF) * want.abs() * 1.01 + LOW[BF] + 4 * LOW[F32]).all()
    dy = torch.randn(6, h, generator=gen).to(BF)
    dx, dw = mg.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=eps)
    want, bound, wdw, bdw = ref.rms_norm_backward(dy, x, w, e)
    most = float(torch.finfo(kind).max)
    dx = dx.cpu().double()
    inside = want.abs() + bound < most / 2                  # (rows of the smallest numbers: gradients past the range)
    # the difference's and r's products below the normal numbers: a step of fp32 each
    assert ((dx - want).abs() <= bound + HALF[kind] * want.abs() * 1.01 + LOW[kind] + 8 * LOW[F32])[inside].all()
    assert ((dw.cpu().double() - wdw).abs() <= bdw + 16 * LOW[F32]).all()


@pytest.mark.parametrize("kind", [BF, F32])
def test_mx_rows_at_the_ends(kind):
    gen = torch.Generator().manual_seed(3)
    x = rows(1024, kind, gen)
    w = torch.rand(1024, generator=gen) + 0.5
    for dtype in ("e4m3", "e5m2", "e2m1x2"):
        codes, sf = mg.rms_norm(x.cuda(), w.cuda(), dtype=dtype)
        want = ref.rms_norm(x, w, torch.tensor(1e-6, dtype=F32).double())
        # scales below 2^-127 do not exist: a block's values there are rounded to the lowest scale's steps
        ref.check_mx(codes, sf, dtype, want, ref.Y_OFF * want.abs() + 4 * LOW[F32])
