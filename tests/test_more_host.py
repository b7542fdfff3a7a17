"""The norm, the router with groups and rows kept in 8 bits without a GPU:
argument rules of the C functions and of the Python front, buffers that may not
overlap, and the float64 reference against differences and by brute force."""
import ctypes
import math
import os

import pytest

torch = pytest.importorskip("torch")

import moe_grouped_block_amd as mg  # noqa: E402
import layer_ref  # noqa: E402
import more_ref as ref  # noqa: E402

OK, INVALID, MISALIGNED, NOT_SUPPORTED = 0, 1, 2, 3
P, APART = 0x7F0000000000, 1 << 36


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


def at(i, off=0):
    return P + i * APART + off


def test_struct_layouts():
    assert ctypes.sizeof(mg.moegg_route_groups) == 12
    assert ctypes.sizeof(mg.moegg_linear_saved) == 32 and mg.moegg_linear_saved.x_sf.offset == 16
    assert ctypes.sizeof(mg.moegg_norm_problem) == 32 and mg.moegg_norm_problem.eps.offset == 28
    assert ctypes.sizeof(mg.moegg_norm_args) == 13 * 8


# ---- the router with groups ---------------------------------------------------------

def _grouped(groups, prob=None, given=True, **ptr):
    p = mg.moegg_route_problem(**{**dict(num_tokens=10, num_experts=64, top_k=6, dtype=5, score=0, renormalise=1, scale=1.0),
                                  **(prob or {})})
    a = {**dict(logits=at(0), bias=None, ids=at(1), weights=at(2)), **ptr}
    return mg._load().moegg_route_grouped(p, mg.moegg_route_groups(*groups) if given else None, a["logits"], a["bias"],
                                          a["ids"], a["weights"], None)


@pytest.mark.parametrize("groups,prob,ptr,want", [
    ((0, 1, 1), {}, {}, INVALID), ((-8, 1, 1), {}, {}, INVALID), ((7, 2, 1), {}, {}, INVALID), ((8, 0, 1), {}, {}, INVALID),
    ((8, 9, 1), {}, {}, INVALID), ((8, 3, 0), {}, {}, INVALID), ((8, 3, 3), {}, {}, INVALID),
    ((32, 2, 1), {}, {}, INVALID),                                   # four experts for six choices
    ((128, 64, 1), dict(num_experts=128), {}, NOT_SUPPORTED),
    ((8, 3, 1), dict(top_k=0), {}, INVALID), ((8, 3, 1), dict(dtype=1), {}, INVALID),
    ((8, 3, 1), {}, dict(ids=None), INVALID), ((8, 3, 1), {}, dict(logits=at(0, 8)), MISALIGNED),
    ((8, 3, 1), {}, dict(ids=at(0, 64)), INVALID),                   # overlaps the logits
    ((8, 3, 1), dict(num_tokens=0), dict(logits=None, ids=None, weights=None), OK),
])
def test_grouped_route_refusals(groups, prob, ptr, want):
    assert _grouped(groups, prob, **ptr) == want, mg.moegg_last_error()


def test_grouped_route_without_groups():
    assert _grouped((8, 3, 1), given=False) == INVALID


def test_reference_groups_by_brute_force():
    """The choice as the best of all sets of groups and experts (no ties)."""
    from itertools import combinations
    gen = torch.Generator().manual_seed(1)
    x, bias = torch.randn(12, 12, generator=gen), torch.randn(12, generator=gen) * 0.2
    ids = ref.route_grouped(x, 3, 4, 2, 2, "sigmoid", bias)
    s = (torch.sigmoid(x.double()) + bias.double()).tolist()
    for t in range(12):
        def score(g):
            return max(s[t][i] + s[t][j] for i, j in combinations(range(3 * g, 3 * g + 3), 2))
        pair = max(combinations(range(4), 2), key=lambda q: score(q[0]) + score(q[1]))
        members = [e for g in pair for e in range(3 * g, 3 * g + 3)]
        best = max(combinations(members, 3), key=lambda q: sum(s[t][e] for e in q))
        assert set(best) == set(ids[t].tolist())


# ---- norm ----------------------------------------------------------------------------

NORM = dict(rows=10, width=512, x_dtype=3, stream_dtype=3, mx_dtype=1, sf_layout=0, eps=1e-6)
NORM_IN = dict(x=10 * 1024, weight=2048)
NORM_OUT = dict(h=10 * 1024, y=10 * 1024, codes=5120, sf=160)


def _norm(prob=None, **ptr):
    a = {n: at(i) for i, n in enumerate([*NORM_IN, *NORM_OUT])}
    a["residual"] = at(9)
    a.update(ptr)
    return mg._load().moegg_rms_norm(mg.moegg_norm_problem(**{**NORM, **(prob or {})}), mg.moegg_norm_args(**a), None)


EMPTY = {n: None for n in ("x", "residual", "weight", "h", "y", "codes", "sf")}


@pytest.mark.parametrize("prob,ptr,want", [
    (dict(rows=-1), {}, INVALID), (dict(rows=1 << 31), {}, NOT_SUPPORTED), (dict(width=0), {}, NOT_SUPPORTED),
    (dict(width=520), {}, NOT_SUPPORTED), (dict(width=516, mx_dtype=0), dict(codes=None, sf=None), NOT_SUPPORTED),
    (dict(width=384, mx_dtype=2), {}, NOT_SUPPORTED), (dict(width=32768 + 128), {}, NOT_SUPPORTED),
    (dict(rows=(1 << 31) - 1, width=32768), {}, NOT_SUPPORTED),
    (dict(x_dtype=1), {}, INVALID), (dict(x_dtype=5), {}, NOT_SUPPORTED), (dict(stream_dtype=4), {}, INVALID),
    (dict(mx_dtype=3), {}, INVALID), (dict(mx_dtype=5), {}, INVALID), (dict(sf_layout=2), {}, INVALID),
    (dict(eps=0.0), {}, INVALID), (dict(eps=-1.0), {}, INVALID), (dict(eps=math.nan), {}, INVALID),
    (dict(eps=math.inf), {}, INVALID),
    ({}, dict(x=None), INVALID), ({}, dict(weight=None), INVALID), ({}, dict(h=None), INVALID), ({}, dict(codes=None), INVALID),
    ({}, dict(sf=None), INVALID), (dict(mx_dtype=0), dict(codes=None, sf=None, y=None), INVALID),
    (dict(mx_dtype=0), {}, INVALID),                                 # codes without their type
    ({}, dict(residual=None), INVALID),                              # h without a residual
    (dict(stream_dtype=5), dict(residual=None, h=None), INVALID),    # x not of the stream's type
    ({}, dict(dy=at(12)), INVALID),
    ({}, dict(x=at(0, 8)), MISALIGNED), ({}, dict(weight=at(1, 2)), MISALIGNED), ({}, dict(sf=at(5, 4)), MISALIGNED),
    ({}, dict(residual=at(9, 2)), MISALIGNED),
    (dict(rows=0), EMPTY, OK),
])
def test_norm_refusals(prob, ptr, want):
    assert _norm(prob, **ptr) == want, mg.moegg_last_error()


def _norm_backward(prob=None, **ptr):
    a = dict(weight=at(0), h=at(1), dy=at(2), dh=at(3), dx=at(4), dweight=at(5), workspace=at(6), workspace_bytes=1 << 30)
    a.update(ptr)
    return mg._load().moegg_rms_norm_backward(mg.moegg_norm_problem(**{**NORM, **(prob or {})}), mg.moegg_norm_args(**a), None)


@pytest.mark.parametrize("prob,ptr,want", [
    (dict(rows=-1), {}, INVALID), (dict(width=516), {}, NOT_SUPPORTED), (dict(width=32776), {}, NOT_SUPPORTED),
    (dict(stream_dtype=1), {}, INVALID), (dict(eps=0.0), {}, INVALID),
    ({}, dict(dx=None, dweight=None), INVALID), ({}, dict(dy=None), INVALID), ({}, dict(h=None), INVALID),
    ({}, dict(workspace=None), INVALID), ({}, dict(workspace_bytes=16), INVALID), ({}, dict(x=at(9)), INVALID),
    ({}, dict(y=at(9)), INVALID), ({}, dict(dx=at(4, 8)), MISALIGNED), ({}, dict(dweight=at(5, 2)), MISALIGNED),
    ({}, dict(dx=at(3, 16)), INVALID), ({}, dict(dweight=at(3)), INVALID),
    (dict(rows=0), dict(dx=None, dweight=None, dy=None, h=None, dh=None, workspace=None), OK),
])
def test_norm_backward_refusals(prob, ptr, want):
    assert _norm_backward(prob, **ptr) == want, mg.moegg_last_error()


def test_norm_workspace():
    lib = mg._load()
    for rows, width in [(1, 8), (5, 2048), (16384, 2048), (100000, 32768), (1 << 30, 8)]:
        need = lib.moegg_rms_norm_backward_workspace(mg.moegg_norm_problem(rows, width, 3, 3, 0, 0, 1e-6))
        assert 4 * width <= need <= 4 * width * 1024
    assert lib.moegg_rms_norm_backward_workspace(mg.moegg_norm_problem(0, 64, 3, 3, 0, 0, 1e-6)) == 0
    assert lib.moegg_rms_norm_backward_workspace(mg.moegg_norm_problem(-1, 64, 3, 3, 0, 0, 1e-6)) == -1


def test_reference_norm_against_differences():
    gen = torch.Generator().manual_seed(1)
    h, w, dy, g = (torch.randn(*s, generator=gen).double() for s in ((4, 24), (24,), (4, 24), (4, 24)))
    dx, _, dw, _ = ref.rms_norm_backward(dy, h, w, 1e-3, g)

    def loss(h, w):
        return float((ref.rms_norm(h, w, 1e-3) * dy).sum() + (h * g).sum())
    d = 1e-6
    for t, grad in ((h, dx), (w, dw)):
        flat, gf = t.reshape(-1), grad.reshape(-1)
        for i in range(0, flat.numel(), 7):
            old = flat[i].item()
            flat[i] = old + d
            up = loss(h, w)
            flat[i] = old - d
            down = loss(h, w)
            flat[i] = old
            assert abs((up - down) / (2 * d) - gf[i].item()) < 1e-7 * max(1.0, abs(gf[i].item()))


# ---- rows in 8 bits -------------------------------------------------------------------

def _quantise(x=at(0), x_dtype=3, rows=10, width=512, dtype=1, layout=0, codes=at(1), sf=at(2)):
    return mg._load().moegg_quantise(x, x_dtype, rows, width, dtype, layout, codes, sf, None)


def _dequantise(x=at(0), x_dtype=3, rows=10, width=512, dtype=1, layout=0, codes=at(1), sf=at(2)):
    return mg._load().moegg_dequantise(codes, sf, rows, width, dtype, layout, x, x_dtype, None)


@pytest.mark.parametrize("f", [_quantise, _dequantise])
@pytest.mark.parametrize("kw,want", [
    (dict(x_dtype=1), INVALID), (dict(dtype=2), INVALID), (dict(dtype=3), INVALID), (dict(layout=2), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), NOT_SUPPORTED), (dict(width=0), NOT_SUPPORTED), (dict(width=48), NOT_SUPPORTED),
    (dict(width=96, layout=1), NOT_SUPPORTED), (dict(width=(1 << 20) + 32), NOT_SUPPORTED),
    (dict(rows=(1 << 31) - 1, width=1 << 20), NOT_SUPPORTED),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(sf=None), INVALID), (dict(x=at(0, 8)), MISALIGNED),
    (dict(codes=at(1, 4)), MISALIGNED), (dict(sf=at(2, 8)), MISALIGNED), (dict(codes=at(0, 10 * 1024 - 16)), INVALID),
    (dict(sf=at(0, 16)), INVALID), (dict(rows=0, x=None, codes=None, sf=None), OK),
])
def test_rows_refusals(f, kw, want):
    assert f(**kw) == want, mg.moegg_last_error()


def test_quantise_outputs_lie_apart():
    assert _quantise(sf=at(1, 5104)) == INVALID and _quantise(codes=at(2), sf=at(2, 16)) == INVALID


# ---- linear from and to 8 bits ----------------------------------------------------------

LIN = dict(m=300, n=256, k=512, num_groups=1, act=7, dtype=3)
SAVED = dict(x_dtype=3, x_sf_layout=0, c_dtype=1, reserved=0, x_sf=None, c_sf=at(5))


def _saving(prob=None, saved=None, **ptr):
    a = dict(x=at(0), w=at(1), bias=at(2), residual=at(3), y=at(4), c=at(6), workspace=at(7), workspace_bytes=1 << 30)
    a.update(ptr)
    return mg._load().moegg_linear_saving(mg.moegg_linear_problem(**{**LIN, **(prob or {})}), mg.moegg_linear_args(**a),
                                          mg.moegg_linear_saved(**{**SAVED, **(saved or {})}), None)


@pytest.mark.parametrize("prob,saved,ptr,want", [
    (dict(n=264), {}, {}, NOT_SUPPORTED), ({}, dict(c_dtype=2), {}, INVALID), ({}, dict(c_dtype=0), {}, INVALID),
    ({}, dict(x_dtype=1, x_sf=at(8)), {}, NOT_SUPPORTED), ({}, dict(c_sf=None), {}, INVALID), ({}, {}, dict(c=None), INVALID),
    ({}, dict(c_dtype=3), {}, INVALID), ({}, dict(reserved=1), {}, INVALID), ({}, dict(x_sf_layout=2), {}, INVALID),
    ({}, dict(x_sf=at(8)), {}, INVALID), ({}, dict(c_sf=at(5, 4)), {}, MISALIGNED),
    ({}, dict(c_sf=at(6, 16)), {}, INVALID), ({}, dict(c_sf=at(4, 16)), {}, INVALID), ({}, dict(c_sf=at(0, 16)), {}, INVALID),
    ({}, dict(c_sf=at(3, 16)), {}, INVALID), ({}, {}, dict(c=at(4, 300 * 512 - 16)), INVALID),
    ({}, {}, dict(c=at(3, 300 * 512 - 16)), INVALID), (dict(k=4096), {}, dict(c=at(7)), INVALID), (dict(k=4096), dict(c_sf=at(7)), {}, INVALID),
    ({}, {}, dict(dy=at(9)), INVALID), (dict(k=4096), {}, dict(workspace=None), INVALID),
    (dict(m=0), dict(c_sf=None), dict(x=None, w=None, y=None, c=None, residual=None, bias=None), OK),
])
def test_saving_refusals(prob, saved, ptr, want):
    assert _saving(prob, saved, **ptr) == want, mg.moegg_last_error()


def _saved_backward(prob=None, saved=None, **ptr):
    a = dict(x=at(0), w=at(1), c=at(2), dy=at(3), dx=at(4), dw=at(5), db=at(6), workspace=at(7), workspace_bytes=1 << 30)
    a.update(ptr)
    s = dict(x_dtype=1, x_sf_layout=1, c_dtype=4, reserved=0, x_sf=at(8), c_sf=at(9))
    return mg._load().moegg_linear_saved_backward(mg.moegg_linear_problem(**{**LIN, **(prob or {})}), mg.moegg_linear_args(**a),
                                                  mg.moegg_linear_saved(**{**s, **(saved or {})}), None)


@pytest.mark.parametrize("prob,saved,ptr,want", [
    (dict(k=520), dict(x_sf_layout=0), {}, NOT_SUPPORTED), (dict(k=544), {}, {}, NOT_SUPPORTED),
    (dict(n=264), {}, {}, NOT_SUPPORTED), ({}, dict(x_dtype=2), {}, INVALID), ({}, dict(x_sf=None), {}, INVALID),
    ({}, dict(c_sf=None), {}, INVALID), ({}, dict(x_dtype=3), {}, INVALID), ({}, dict(reserved=7), {}, INVALID),
    ({}, dict(x_sf=at(8, 2)), {}, MISALIGNED), ({}, {}, dict(c=None), INVALID), ({}, {}, dict(x=None), INVALID),
    ({}, dict(x_sf=at(4, 64)), {}, INVALID), ({}, dict(c_sf=at(5, 64)), {}, INVALID), ({}, {}, dict(x=at(4, 64)), INVALID),
    ({}, {}, dict(workspace_bytes=1 << 10), INVALID), ({}, {}, dict(dx=at(0, 300 * 512 - 16)), INVALID),
    ({}, dict(x_sf=at(7, 64)), {}, INVALID), ({}, dict(c_sf=at(7, 64)), {}, INVALID),
])
def test_saved_backward_refusals(prob, saved, ptr, want):
    assert _saved_backward(prob, saved, **ptr) == want, mg.moegg_last_error()


def test_saved_workspaces():
    """x's BF16 form is part of the workspace only where dw needs one of an x in 8 bits."""
    lib, p = mg._load(), mg.moegg_linear_problem(3000, 256, 512, 1, 7, 3)
    plain, x8 = mg.moegg_linear_saved(3, 0, 3), mg.moegg_linear_saved(1, 0, 3)
    for want in range(1, 8):
        base = lib.moegg_linear_backward_workspace(p, want)
        assert lib.moegg_linear_saved_backward_workspace(p, plain, want) == base
        more = lib.moegg_linear_saved_backward_workspace(p, x8, want) - base
        assert more >= 3000 * 512 * 2 if want & 2 else more == 0
    # the largest tiles of dw read the codes themselves
    big = mg.moegg_linear_problem(16384, 2816, 2048, 1, 1, 3)
    assert lib.moegg_linear_saved_backward_workspace(big, x8, 7) == lib.moegg_linear_backward_workspace(big, 7)
    assert lib.moegg_linear_saving_workspace(p, plain) == lib.moegg_linear_workspace(p)
    assert lib.moegg_linear_saving_workspace(p, mg.moegg_linear_saved(3, 0, 2)) == -1
    assert lib.moegg_linear_saved_backward_workspace(p, mg.moegg_linear_saved(1, 0, 3, 5), 7) == -1


# ---- the front -------------------------------------------------------------------------

def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


F32, U8 = torch.float32, torch.uint8


@pytest.mark.parametrize("call,error", [
    (lambda: mg.rms_norm(torch.ones(2, 64, dtype=torch.bfloat16), torch.ones(64)), ValueError),          # not on a GPU
    (lambda: mg.rms_norm([1], torch.ones(64)), TypeError),
    (lambda: mg.rms_norm(meta(2, 64, dtype=torch.float16), meta(64, dtype=F32)), TypeError),
    (lambda: mg.rms_norm_backward(meta(2, 64), meta(2, 64), meta(64, dtype=F32), need=()), ValueError),
    (lambda: mg.rms_norm_backward(meta(2, 64), meta(2, 64), meta(64, dtype=F32), need=("dx", "dh")), ValueError),
    (lambda: mg.dequantise(meta(2, 64)), TypeError),
    (lambda: mg.dequantise((meta(2, 64, dtype=U8),)), TypeError),
    (lambda: mg.quantise(torch.ones(2, 64)), ValueError),
    (lambda: mg.linear_backward(meta(2, 64), meta(2, 64), meta(64, 64), x_dtype="e4m3"), TypeError),
    (lambda: mg.linear_backward(meta(2, 64), (meta(2, 64), meta(2, 2)), meta(64, 64), x_dtype="e3m4"), ValueError),
])
def test_front_refusals(call, error):
    with pytest.raises(error):
        call()


@pytest.fixture()
def front(monkeypatch):
    """The front with its checks of place taken for passed, and no call behind it."""
    def enqueued(*_):
        raise AssertionError("the call went through")
    monkeypatch.setattr(mg.layer, "_lead", lambda t, *_: 0)
    monkeypatch.setattr(mg.layer, "_want", lambda *_: 0)
    monkeypatch.setattr(mg.layer, "_on", enqueued)


@pytest.mark.parametrize("call", [
    lambda: mg.rms_norm(meta(1, 64), meta(64), dtype="f16"), lambda: mg.rms_norm(meta(1, 64), meta(64), copy="bf16"),
    lambda: mg.rms_norm(meta(1, 64), meta(64), dtype="e4m3", copy="e4m3"),
    lambda: mg.rms_norm(meta(1, 64), meta(64), h=meta(1, 64)), lambda: mg.rms_norm(meta(1, 64), meta(64), sf_layout="planes"),
    lambda: mg.rms_norm(meta(1, 2 ** 32 + 64), meta(64)), lambda: mg.rms_norm_backward(meta(1, 64), meta(1, 2 ** 32 + 64), meta(64)),
    lambda: mg.quantise(meta(1, 64), dtype="e2m1x2"), lambda: mg.quantise(meta(1, 64), dtype="bf16"),
    lambda: mg.quantise(meta(1, 2 ** 32 + 64)), lambda: mg.dequantise((meta(1, 2 ** 32 + 64), None)),
    lambda: mg.dequantise((meta(1, 64), meta(1, 2)), to="e4m3"), lambda: mg.linear(meta(1, 64), meta(64, 64), save_c="e2m1x2"),
    lambda: mg.linear_backward(meta(1, 64), meta(1, 64), meta(64, 64), c=(meta(1, 64), meta(1, 2)), c_dtype="fp8"),
    lambda: mg.route(meta(1, 64), 2, num_groups=2 ** 32 + 8, top_groups=2), lambda: mg.route(meta(1, 64), 2, top_groups=-1),
])
def test_front_refuses_names_and_sizes(front, call):
    with pytest.raises(ValueError):
        call()


def test_front_passes_what_is_right(front):
    for call in (lambda: mg.rms_norm(meta(1, 128), meta(128), copy="e4m3"), lambda: mg.quantise(meta(1, 64), dtype="e5m2"),
                 lambda: mg.route(meta(1, 64), 2, num_groups=8, top_groups=2),
                 lambda: mg.linear(meta(1, 64), meta(64, 64), save_c="e4m3")):
        with pytest.raises(AssertionError, match="went through"):
            call()


def test_reference_decodes_what_it_encodes():
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(9, 256, generator=gen).double()
    for fmt in ("e4m3", "e5m2", "e2m1x2"):
        codes, byte = layer_ref.mx_encode(x, fmt)
        # within half a step of the grid (relative, and of its lowest step below)
        v = ref.check_mx(torch.from_numpy(codes), torch.from_numpy(byte), fmt, x, 0.0 * x)
        again, b2 = layer_ref.mx_encode(v, fmt)
        assert (torch.from_numpy(b2) <= torch.from_numpy(byte)).all()
        assert torch.equal(ref.decode(again, b2, fmt), v)
