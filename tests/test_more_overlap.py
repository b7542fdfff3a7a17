"""No output of the norm, the grouped router, the rows in 8 bits or linear from
and to 8 bits may share memory with an input, a workspace or another output:
every pair, through the C functions on fake pointers (no GPU: a refused call
enqueues nothing)."""
import os

import pytest

pytest.importorskip("torch")
import moe_grouped_block_amd as mg  # noqa: E402

INVALID = 1
BASE, APART = 0x7F0000000000, 1 << 36


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


def route_grouped(**p):
    q = mg.moegg_route_problem(100, 64, 6, 5, 0, 1, 1.0)
    return mg._load().moegg_route_grouped(q, mg.moegg_route_groups(8, 3, 2), p["logits"], p["bias"], p["ids"], p["weights"], None)


def rms_norm(**p):
    return mg._load().moegg_rms_norm(mg.moegg_norm_problem(100, 512, 3, 5, 1, 0, 1e-6), mg.moegg_norm_args(**p), None)


def rms_norm_backward(**p):
    q = mg.moegg_norm_problem(100, 512, 3, 5, 0, 0, 1e-6)
    assert mg._load().moegg_rms_norm_backward_workspace(q) >= 256
    return mg._load().moegg_rms_norm_backward(q, mg.moegg_norm_args(**p, workspace_bytes=1 << 30), None)


def quantise(**p):
    return mg._load().moegg_quantise(p["x"], 3, 100, 512, 1, 0, p["codes"], p["sf"], None)


def dequantise(**p):
    return mg._load().moegg_dequantise(p["codes"], p["sf"], 100, 512, 1, 0, p["x"], 3, None)


def linear_saving(**p):
    q, sf = mg.moegg_linear_problem(300, 256, 4096, 1, 0, 3), p.pop("c_sf")
    k = mg.moegg_linear_saved(3, 0, 1, 0, None, sf)
    assert mg._load().moegg_linear_saving_workspace(q, k) > 256
    return mg._load().moegg_linear_saving(q, mg.moegg_linear_args(**p, workspace_bytes=1 << 30), k, None)


def linear_saved_backward(**p):
    q = mg.moegg_linear_problem(300, 256, 512, 2, 7, 3)
    k = mg.moegg_linear_saved(1, 0, 4, 0, p.pop("x_sf"), p.pop("c_sf"))
    assert mg._load().moegg_linear_saved_backward_workspace(q, k, 7) > 300 * 1024
    return mg._load().moegg_linear_saved_backward(q, mg.moegg_linear_args(**p, workspace_bytes=1 << 30), k, None)


# function: its inputs, what it writes, and the sizes in bytes of all of them
CALLS = {
    route_grouped: (dict(logits=100 * 64 * 4, bias=64 * 4), dict(ids=2400, weights=2400)),
    rms_norm: (dict(x=100 * 1024, residual=100 * 2048, weight=2048), dict(h=100 * 2048, y=100 * 1024, codes=100 * 512, sf=1600)),
    rms_norm_backward: (dict(weight=2048, h=100 * 2048, dy=100 * 1024, dh=100 * 2048),
                        dict(dx=100 * 2048, dweight=2048, workspace=256)),
    quantise: (dict(x=100 * 1024), dict(codes=100 * 512, sf=1600)),
    dequantise: (dict(codes=100 * 512, sf=1600), dict(x=100 * 1024)),
    linear_saving: (dict(x=300 * 4096 * 2, w=256 * 4096 * 2, bias=1024, residual=300 * 512),
                    dict(y=300 * 512, c=300 * 256, c_sf=300 * 8, workspace=256)),
    linear_saved_backward: (dict(x=300 * 512, w=2 * 256 * 1024, offsets=8, c=300 * 256, dy=300 * 512, x_sf=300 * 16, c_sf=300 * 8),
                            dict(dx=300 * 1024, dw=2 * 256 * 1024, db=2048, workspace=256)),
}
PAIRS = [(f, a, b) for f, (ins, outs) in CALLS.items()
         for i, b in enumerate(outs) for a in [*ins, *list(outs)[:i]]]


@pytest.mark.parametrize("f,a,b", PAIRS, ids=[f"{f.__name__}-{a}-{b}" for f, a, b in PAIRS])
def test_outputs_lie_apart(f, a, b):
    ins, outs = CALLS[f]
    size = {**ins, **outs}
    at = {name: BASE + i * APART for i, name in enumerate(size)}
    # b ends in a's first 16 bytes, or begins in a's last ones
    for where in (at[a] - size[b] // 16 * 16 + (16 if size[b] % 16 == 0 else 0), at[a] + (size[a] - 1) // 16 * 16):
        assert where < at[a] + size[a] and at[a] < where + size[b] and where % 16 == 0
        assert f(**{**at, b: where}) == INVALID, (f.__name__, a, b)
        assert "overlap" in mg.moegg_last_error()


def test_tensors_without_elements_share_nothing():
    """An empty tensor's address may lie anywhere, also inside another tensor."""
    lib = mg._load()
    assert lib.moegg_quantise(BASE, 3, 0, 512, 1, 0, BASE + 16, BASE, None) == 0
    assert lib.moegg_dequantise(BASE, BASE, 0, 512, 1, 0, BASE + 64, 3, None) == 0
    q = mg.moegg_norm_problem(0, 512, 3, 3, 1, 0, 1e-6)
    assert lib.moegg_rms_norm(q, mg.moegg_norm_args(*[BASE] * 7), None) == 0
    assert lib.moegg_rms_norm_backward(q, mg.moegg_norm_args(weight=BASE + APART, h=BASE, dy=BASE, dh=BASE, dx=BASE + 16), None) == 0
