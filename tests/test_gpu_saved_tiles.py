"""GPU tests of linear that keeps c in 8 bits and of its gradients from 8 bits on
the largest tiles: dw's reads of the codes, with its sums whole and in parts,
and y beside a kept c bit for bit.  The path that a shape is here for is stated
by the workspaces' sizes, on the host."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ACTS = {"none": 0, "swiglu": 1, "srelu": 2, "gelu": 7}
KINDS = {"e4m3": 1, "e5m2": 4}


def dw_path(m, n, k, act, fmt, layout, dw_dtype):
    """Whether dw reads x's codes itself (no BF16 copy of x in the workspace), and whether its sums are split (parts
    in the workspace beside dz)."""
    lib, p = mg._load(), mg.moegg_linear_problem(m, n, k, 1, ACTS[act], 5 if dw_dtype == "f32" else 3)
    keep = mg.moegg_linear_saved(KINDS[fmt], int(layout == "kplanes"), 3)
    plain = lib.moegg_linear_backward_workspace(p, 2)
    dz = 0 if act == "none" else -(-m * n * 2 // 256) * 256
    return lib.moegg_linear_saved_backward_workspace(p, keep, 2) == plain, plain > dz


@pytest.mark.parametrize("m,n,k,act,fmt,layout,split", [
    (16384, 2816, 2048, "swiglu", "e4m3", "row_major", True), (16384, 2816, 2048, "swiglu", "e5m2", "kplanes", True),
    (16381, 2816, 2080, "swiglu", "e4m3", "row_major", True), (16381, 2816, 2080, "swiglu", "e5m2", "row_major", True),
    (8191, 2080, 2080, "srelu", "e5m2", "row_major", True),       # widths that end inside a tile, three parts
    (8161, 2048, 2176, "gelu", "e4m3", "kplanes", True),
    (16381, 1408, 2048, "none", "e4m3", "kplanes", True),         # five parts
    (4096, 4096, 4096, "gelu", "e4m3", "kplanes", False), (4093, 4096, 4096, "srelu", "e5m2", "row_major", False),
    (600, 1056, 8192, "gelu", "e4m3", "kplanes", False)])
@pytest.mark.parametrize("need,dw_dtype", [(("dx", "dw", "db"), "bf16"), (("dw",), "f32")])
def test_dw_from_codes(m, n, k, act, fmt, layout, split, need, dw_dtype):
    """Bit for bit as from the same values in BF16: parts of the rows that begin inside x and end where rows
    follow, their join, ragged last steps."""
    assert dw_path(m, n, k, act, fmt, layout, dw_dtype) == (True, split)
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    x8 = mg.quantise(torch.randn(m, k, generator=gen, device="cuda"), dtype=fmt, sf_layout=layout)
    c8 = None if act == "none" else mg.quantise(torch.randn(m, n, generator=gen, device="cuda"), dtype=fmt)
    w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(BF)
    dy = torch.randn(m, n // 2 if act == "swiglu" else n, generator=gen, device="cuda").to(BF)
    print(f"[gpu-case] dw from codes m={m} n={n} k={k} {act} {fmt} {layout} {need} {dw_dtype}", flush=True)
    got = mg.linear_backward(dy, x8, w, c=c8, act=act, need=need, dw_dtype=dw_dtype, x_dtype=fmt, c_dtype=fmt, sf_layout=layout)
    x = mg.dequantise(x8, dtype=fmt, sf_layout=layout)
    c = None if c8 is None else mg.dequantise(c8, dtype=fmt)
    same = mg.linear_backward(dy, x, w, c=c, act=act, need=need, dw_dtype=dw_dtype)
    for a, b in zip(got, same):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    if act == "none":
        # float64, a product of two bf16 numbers being exact in fp32: m roundings of the sum, and one of the result
        xd, d = x.double(), dy.double()
        want, mag = d.t() @ xd, d.abs().t() @ xd.abs()
        eps = 2.0 ** -24 if dw_dtype == "f32" else 2.0 ** -8
        assert ((got[1].double() - want).abs() <= (m + 16) * 2.0 ** -24 * mag + eps * want.abs() * 1.01).all()


@pytest.mark.parametrize("layout", ["row_major", "kplanes"])
def test_not_numbers_stay_in_their_part(layout):
    """A scale byte of 255 in the first row of dw's second part of r: NaN in its 32 columns alone."""
    m, n, k = 16384, 2816, 2048
    assert dw_path(m, n, k, "none", "e4m3", layout, "bf16") == (True, True)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x8 = mg.quantise(torch.randn(m, k, generator=gen, device="cuda"), sf_layout=layout)
    dy = torch.randn(m, n, generator=gen, device="cuda").to(BF)
    w = torch.zeros(n, k, dtype=BF, device="cuda")
    for row, block in ((m // 2, 5), (m // 2 - 1, 63), (m - 1, 0)):
        at = (block // 4, row, block % 4) if layout == "kplanes" else (row, block)
        old = x8[1][at].item()
        x8[1][at] = 255
        _, dw, _ = mg.linear_backward(dy, x8, w, need=("dw",), x_dtype="e4m3", sf_layout=layout)
        x8[1][at] = old
        nan = torch.isnan(dw)
        assert nan[:, 32 * block:32 * block + 32].all() and int(nan.sum()) == 32 * n


@pytest.mark.parametrize("m,n,k,act,groups,split", [
    (4096, 2816, 2048, "swiglu", 0, False), (3000, 2048, 1408, "swiglu", 0, False),        # 256 x 256 and 128 x 128, whole
    (2500, 2048, 8192, "swiglu", 0, True), (4096, 4160, 2048, "gelu", 0, True),            # 256 x 256, all and the last in parts
    (2304, 4096, 4096, "srelu", 0, True), (600, 1056, 8192, "gelu", 0, True),              # 128 x 128
    (300, 160, 4096, "none", 0, True), (193, 2816, 2048, "swiglu", 0, False), (100, 96, 264, "gelu", 0, False),   # 64 x 64
    (5000, 2048, 520, "swiglu", 6, False), (3001, 1056, 2048, "gelu", 20, False), (777, 2816, 264, "srelu", 64, False)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype,residual", [("bf16", False), ("f32", True)])
def test_y_beside_a_kept_c(m, n, k, act, groups, split, fmt, dtype, residual):
    """Keeping c in 8 bits leaves y as it is, bit for bit, where the tiles are the same (no rows of either call go by the
    kernel for few rows), and c is what its fp32 values give: their BF16 form is off by a rounding."""
    lib, p = mg._load(), mg.moegg_linear_problem(m, n, k, max(groups, 1), ACTS[act], 5 if dtype == "f32" else 3)
    need = lib.moegg_linear_saving_workspace(p, mg.moegg_linear_saved(3, 0, KINDS[fmt]))
    assert need == lib.moegg_linear_workspace(p) and (need > 0) == split
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.randn(m, k, generator=gen, device="cuda").to(BF)
    w = (torch.randn(*((groups, n, k) if groups else (n, k)), generator=gen, device="cuda") / math.sqrt(k)).to(BF)
    b = torch.randn(*((groups, n) if groups else (n,)), generator=gen, device="cuda") * 0.3
    res = torch.randn(m, n // 2 if act == "swiglu" else n, generator=gen, device="cuda").to(BF) if residual else None
    off = None
    if groups:
        cut = torch.sort(torch.randint(0, m + 1, (groups - 1,), generator=gen, device="cuda")).values.tolist()
        off = torch.tensor(cut + [m], dtype=torch.int32, device="cuda")
    print(f"[gpu-case] y beside c in {fmt} m={m} n={n} k={k} {act} groups={groups} {dtype}", flush=True)
    how = dict(bias=b, act=act, residual=res, offsets=off, dtype=dtype)
    y0, c0 = mg.linear(x, w, save_c=True, **how)
    y1 = mg.linear(x, w, **how)
    y, (codes, sf) = mg.linear(x, w, save_c=fmt, **how)
    assert torch.equal(y, y0) and torch.equal(y, y1)
    # a block's values in 8 bits of its BF16 ones are half a step away at most, and BF16's rounding more
    back, c = mg.dequantise((codes, sf), dtype=fmt, to="f32").double(), c0.double()
    rel, low = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}[fmt]
    scale = torch.exp2(sf.double() - 127.0).repeat_interleave(32, 1)
    most = c.abs() / (1.0 - 2.0 ** -8)
    assert ((back - c).abs() <= torch.maximum(rel * most, low * scale) + 2.0 ** -8 * c.abs() * 1.01).all()
