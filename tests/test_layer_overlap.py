"""No output of a layer operator may share memory with an input, a workspace
or another output: every pair, through the C functions on fake pointers (no
GPU: a refused call enqueues nothing)."""
import ctypes
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


def route(**p):
    q = mg.moegg_route_problem(100, 64, 6, 5, 0, 1, 1.0)
    return mg._load().moegg_route(q, p["logits"], p["bias"], p["ids"], p["weights"], None)


def route_backward(**p):
    q = mg.moegg_route_problem(100, 64, 6, 5, 0, 1, 1.0)
    return mg._load().moegg_route_backward(q, p["logits"], p["ids"], p["dweights"], p["dlogits"], None)


def sort(**p):
    q = mg.moegg_sort_problem(1000, 6, 64, 1, 6000)
    return mg._load().moegg_sort(q, p["ids"], p["weights"], p["padded_offsets"], p["row_of"], p["slot_of"], p["prob"],
                                 p["workspace"], 1 << 20, None)


def dispatch(**p):
    q = mg.moegg_exchange_problem(100, 600, 6, 64, 512, 1, 0)
    return mg._load().moegg_dispatch(q, p["x"], p["row_of"], p["slot_of"], p["padded_offsets"], p["out"], p["sf"], None)


def combine(**p):
    q = mg.moegg_exchange_problem(100, 600, 6, 64, 512, 3, 0)
    return mg._load().moegg_combine(q, p["rows_in"], p["row_of"], p["weights"], p["residual"], p["y"], None)


def combine_backward(**p):
    q = mg.moegg_exchange_problem(100, 600, 6, 64, 512, 1, 0)
    return mg._load().moegg_combine_backward(q, p["dy"], p["row_of"], p["slot_of"], p["padded_offsets"], p["rows_in"],
                                             p["weights"], p["out"], p["sf"], p["dweights"], None)


def unsort(**p):
    return mg._load().moegg_unsort(p["rows_values"], p["row_of"], p["values"], 600, 700, None)


def linear(**p):
    q = mg.moegg_linear_problem(300, 256, 4096, 1, 0, 3)       # (a product whose r is split: it has a workspace)
    assert mg._load().moegg_linear_workspace(q) > 256
    return mg._load().moegg_linear(q, mg.moegg_linear_args(**p, workspace_bytes=1 << 30), None)


def linear_backward(**p):
    q = mg.moegg_linear_problem(300, 256, 512, 2, 7, 3)
    assert mg._load().moegg_linear_backward_workspace(q, 7) > 256
    return mg._load().moegg_linear_backward(q, mg.moegg_linear_args(**p, workspace_bytes=1 << 30), None)


# function: its inputs, what it writes, and the sizes in bytes of all of them
CALLS = {
    route: (dict(logits=100 * 64 * 4, bias=64 * 4), dict(ids=2400, weights=2400)),
    route_backward: (dict(logits=100 * 64 * 4, ids=2400, dweights=2400), dict(dlogits=100 * 64 * 4)),
    sort: (dict(ids=24000, weights=24000), dict(padded_offsets=256, row_of=24000, slot_of=24000, prob=24000, workspace=1536)),
    dispatch: (dict(x=102400, row_of=2400, slot_of=2400, padded_offsets=256), dict(out=307200, sf=9600)),
    combine: (dict(rows_in=614400, row_of=2400, weights=2400, residual=102400), dict(y=102400)),
    combine_backward: (dict(dy=102400, row_of=2400, slot_of=2400, padded_offsets=256, rows_in=614400, weights=2400),
                       dict(out=307200, sf=9600, dweights=2400)),
    unsort: (dict(rows_values=2800, row_of=2400), dict(values=2400)),
    linear: (dict(x=300 * 4096 * 2, w=256 * 4096 * 2, bias=1024, residual=300 * 512),
             dict(y=300 * 512, c=300 * 512, workspace=256)),
    linear_backward: (dict(x=300 * 1024, w=2 * 256 * 1024, offsets=8, c=300 * 512, dy=300 * 512),
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
    lib, e = mg._load(), mg.moegg_exchange_problem(0, 600, 6, 64, 512, 3, 0)
    assert lib.moegg_dispatch(e, BASE + 64, None, BASE, BASE + APART, BASE, None, None) == 0
    assert lib.moegg_combine(e, BASE, None, None, None, BASE + 64, None) == 0
