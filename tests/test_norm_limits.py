"""How many rows rms_norm takes: as many as one launch holds (2^32 threads),
which for narrow rows is several rows a wave.  No GPU: a call whose sizes pass is
refused for a pointer that is not aligned."""
import os

import pytest

pytest.importorskip("torch")

import moe_grouped_block_amd as mg  # noqa: E402

MISALIGNED, NOT_SUPPORTED = 2, 3
BASE, APART = 0x7F0000000000, 1 << 44


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


def threads(rows, width, stream, mx):
    """Threads of the launch: a lane has 8 columns of a BF16 stream, 4 of an fp32 one; 1024 columns are a
    wave's (2048 past 16384 columns); a row has a power of two of lanes, at least 8 (of MX rows 128 columns'
    worth) and a power of two of waves; workgroups are four waves or a row's."""
    unit = 4 if stream == 5 else 8
    lanes = 8 if mx == 0 else 128 // unit
    while lanes < 64 and lanes * unit < width:
        lanes *= 2
    pieces, most = -(-width // (64 * unit)), (1024 if width <= 16384 else 2048) // (64 * unit)
    p = 1
    while p < most and p < pieces:
        p *= 2
    waves = 1
    while p * waves < pieces:
        waves *= 2
    rows_a_group = 64 // lanes * 4 if waves == 1 else max(1, 4 // waves)
    return -(-rows // rows_a_group) * 64 * max(4, waves)


def status(rows, width, stream, mx):
    p = mg.moegg_norm_problem(rows, width, 3, stream, mx, 0, 1e-6)
    a = {n: BASE + i * APART for i, n in enumerate(("weight", "residual", "h", "y"))}
    if mx:
        a["codes"], a["sf"] = BASE + 4 * APART, BASE + 5 * APART
    return mg._load().moegg_rms_norm(p, mg.moegg_norm_args(x=BASE + 6 * APART + 8, **a), None)


@pytest.mark.parametrize("width,stream,mx", [(8, 3, 0), (64, 3, 0), (64, 5, 0), (72, 3, 0), (128, 3, 1), (128, 5, 4), (256, 3, 2),
                                             (256, 5, 2), (264, 3, 0), (512, 3, 0), (520, 5, 0), (1024, 3, 1), (2048, 3, 0),
                                             (2048, 5, 1), (4096, 3, 0), (8200, 3, 0), (16384, 5, 0), (16392, 3, 0), (32768, 5, 1)])
def test_rows_up_to_what_a_launch_holds(width, stream, mx):
    most = 2 ** 32 - 1024
    low, high = 1, 2 ** 31                     # the largest number of rows whose launch holds them
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (mid, high) if threads(mid, width, stream, mx) <= most else (low, mid)
    assert status(low, width, stream, mx) == MISALIGNED, mg.moegg_last_error()
    assert status(low + 1, width, stream, mx) == NOT_SUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("stream,h", [("bf16", 8), ("f32", 8), ("bf16", 64)])
def test_many_narrow_rows(stream, h):
    """2^25 rows and more (a thread count of 2^32 if each had a wave and its place)."""
    torch = pytest.importorskip("torch")
    import more_ref as ref
    t = (1 << 26) + 5
    kind = torch.bfloat16 if stream == "bf16" else torch.float32
    x = torch.zeros(t, h, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(t, h, dtype=kind, device="cuda")
    for at in (0, (1 << 25) - 1, 1 << 25, t - 1):
        x[at] = torch.arange(h, device="cuda").add(at % 7 + 1).to(torch.bfloat16)
    w = torch.linspace(0.5, 1.5, h, device="cuda")
    print(f"[gpu-case] rms_norm {t}x{h} stream={kind}", flush=True)
    y, s = mg.rms_norm(x, w, residual=r, h=r)
    assert s is r and torch.equal(s, x.to(kind))
    live = [0, (1 << 25) - 1, 1 << 25, t - 1]
    want = ref.rms_norm(x[live].cpu(), w.cpu(), 1e-6)
    assert ((y[live].cpu().double() - want).abs() <= (ref.BF16 + ref.Y_OFF) * 1.01 * want.abs()).all()
    y[live] = 0
    assert not y.any()
