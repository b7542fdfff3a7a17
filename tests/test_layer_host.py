"""Layer operators without a GPU: argument rules of the C functions and of the
Python front (nothing is enqueued by a refused call; the pointers below are
fake), sizes of buffers, and the float64 reference against differences."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

import moe_grouped_block_amd as mg  # noqa: E402
import layer_ref as ref  # noqa: E402

OK, INVALID, MISALIGNED, NOT_SUPPORTED = 0, 1, 2, 3
P = 0x7F0000000000           # 16-byte aligned, never dereferenced
FAR = 1 << 40                # keeps fake tensors apart


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


def at(i, off=0):
    return P + i * FAR // 8 + off


# ---- struct layouts as in the header ------------------------------------------

def test_struct_layouts():
    assert ctypes.sizeof(mg.moegg_route_problem) == 32
    assert mg.moegg_route_problem.scale.offset == 28
    assert ctypes.sizeof(mg.moegg_sort_problem) == 32 and mg.moegg_sort_problem.rows.offset == 24
    assert ctypes.sizeof(mg.moegg_exchange_problem) == 40 and mg.moegg_exchange_problem.sf_layout.offset == 32
    assert ctypes.sizeof(mg.moegg_linear_problem) == 32 and mg.moegg_linear_problem.dtype.offset == 24
    assert ctypes.sizeof(mg.moegg_linear_args) == 13 * 8


# ---- refusals of the C functions -------------------------------------------------

def _route(prob=None, **ptr):
    p = dict(num_tokens=10, num_experts=64, top_k=6, dtype=3, score=0, renormalise=1, scale=1.0, **{})
    p.update(prob or {})
    a = dict(logits=at(0), bias=None, ids=at(1), weights=at(2))
    a.update(ptr)
    return mg._load().moegg_route(ctypes.byref(mg.moegg_route_problem(**p)), a["logits"], a["bias"], a["ids"],
                                  a["weights"], None)


@pytest.mark.parametrize("prob,ptr,want", [
    (dict(num_tokens=-1), {}, INVALID), (dict(num_experts=0), {}, INVALID), (dict(num_experts=1025), {}, INVALID),
    (dict(top_k=0), {}, INVALID), (dict(top_k=65), {}, INVALID), (dict(top_k=33), {}, NOT_SUPPORTED),
    (dict(dtype=1), {}, INVALID), (dict(score=2), {}, INVALID), (dict(renormalise=2), {}, INVALID),
    (dict(scale=float("nan")), {}, INVALID), (dict(scale=float("inf")), {}, INVALID),
    (dict(num_tokens=1 << 31), {}, NOT_SUPPORTED),
    ({}, dict(logits=None), INVALID), ({}, dict(ids=None), INVALID), ({}, dict(weights=None), INVALID),
    ({}, dict(logits=at(0, 8)), MISALIGNED), ({}, dict(ids=at(1, 2)), MISALIGNED), ({}, dict(bias=at(3, 1)), MISALIGNED),
    (dict(num_tokens=0), dict(logits=None, ids=None, weights=None), OK),
])
def test_route_refusals(prob, ptr, want):
    assert _route(prob, **ptr) == want, mg.moegg_last_error()


def test_route_backward_refusals():
    lib = mg._load()
    p = mg.moegg_route_problem(num_tokens=10, num_experts=64, top_k=6, dtype=5, score=0, renormalise=1, scale=1.0)
    b = ctypes.byref(p)
    assert lib.moegg_route_backward(b, at(0), at(1), None, at(3), None) == INVALID
    assert lib.moegg_route_backward(b, at(0), at(1), at(2), at(0), None) == INVALID          # in place
    assert lib.moegg_route_backward(b, at(0), at(1), at(2), at(0, 10 * 64 * 4 - 16), None) == INVALID
    assert lib.moegg_route_backward(b, at(0), at(1), at(2), at(3, 8), None) == MISALIGNED
    assert lib.moegg_route_backward(None, at(0), at(1), at(2), at(3), None) == INVALID


def _sort(prob=None, weights=None, probs=None, ws=None, ws_bytes=0, offsets=at(1), slot_of=at(3), row_of=at(2)):
    p = dict(num_tokens=10, top_k=6, num_experts=64, m_aligned=128, rows=60 * 128)
    p.update(prob or {})
    return mg._load().moegg_sort(ctypes.byref(mg.moegg_sort_problem(**p)), at(0), weights, offsets, row_of, slot_of,
                                 probs, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(prob=dict(num_tokens=-1)), INVALID), (dict(prob=dict(top_k=0)), INVALID),
    (dict(prob=dict(top_k=33)), NOT_SUPPORTED), (dict(prob=dict(num_experts=0)), INVALID),
    (dict(prob=dict(num_experts=1025)), INVALID), (dict(prob=dict(m_aligned=0)), INVALID),
    (dict(prob=dict(m_aligned=65537)), INVALID), (dict(prob=dict(rows=60 * 128 - 1)), INVALID),   # too few rows
    (dict(prob=dict(rows=1 << 31)), INVALID),
    (dict(prob=dict(num_tokens=1 << 29)), NOT_SUPPORTED),
    (dict(weights=at(5)), INVALID), (dict(probs=at(5)), INVALID),                                # only one of the two
    (dict(offsets=None), INVALID), (dict(slot_of=None), INVALID), (dict(row_of=at(2, 2)), MISALIGNED),
    (dict(prob=dict(num_tokens=10000, rows=1 << 30)), INVALID),                                  # no workspace
    (dict(prob=dict(num_tokens=10000, rows=1 << 30), ws=at(6), ws_bytes=4), INVALID),
])
def test_sort_refusals(kw, want):
    assert _sort(**kw) == want, mg.moegg_last_error()


def test_sort_sizes():
    lib = mg._load()

    def rows(t, k, e, ma):
        return mg.sort_rows(t, k, e, ma)
    assert rows(1, 6, 64, 128) == 6 * 128              # six experts with one row each
    assert rows(0, 6, 64, 128) == 0
    assert rows(16384, 6, 64, 1) == 98304
    assert rows(16384, 6, 64, 128) == (98304 + 64 * 127) // 128 * 128
    # the bound is reached: every expert one row over a multiple
    assert rows(3 * 65, 1, 3, 64) == 3 * 128
    for t, k, e in [(1, 1, 1), (16384, 6, 64), (1 << 20, 8, 1024), (1 << 24, 32, 4)]:
        p = mg.moegg_sort_problem(num_tokens=t, top_k=k, num_experts=e, m_aligned=1)
        need = lib.moegg_sort_workspace(ctypes.byref(p))
        assert 0 <= need <= 257 * e * 4
    with pytest.raises(mg.MoeggError):
        mg.sort_rows(1 << 28, 8, 64, 128)
    with pytest.raises(mg.MoeggError):
        mg.sort_rows(10, 0, 64, 128)


def _exchange(**over):
    p = dict(num_tokens=10, rows=7680, top_k=6, num_experts=64, width=512, dtype=3, sf_layout=0)
    p.update(over)
    return ctypes.byref(mg.moegg_exchange_problem(**p))


@pytest.mark.parametrize("over,want", [
    (dict(num_tokens=-1), INVALID), (dict(rows=-1), INVALID), (dict(top_k=0), INVALID), (dict(top_k=33), NOT_SUPPORTED),
    (dict(num_experts=0), INVALID), (dict(rows=1 << 31), NOT_SUPPORTED), (dict(dtype=5), INVALID),
    (dict(width=0), NOT_SUPPORTED), (dict(width=516), NOT_SUPPORTED), (dict(width=520, dtype=1), NOT_SUPPORTED),
    (dict(width=384, dtype=2), NOT_SUPPORTED), (dict(width=(1 << 20) + 8), NOT_SUPPORTED), (dict(sf_layout=2), INVALID),
    (dict(dtype=1), INVALID),                                                                    # MX rows without scales
])
def test_dispatch_refusals(over, want):
    assert mg._load().moegg_dispatch(_exchange(**over), at(0), at(1), at(2), at(3), at(4), None, None) == want, \
        mg.moegg_last_error()


def test_exchange_pointer_refusals():
    lib, e = mg._load(), _exchange()
    assert lib.moegg_dispatch(e, at(0), at(1), at(2), at(3), at(4), at(5), None) == INVALID      # scales with bf16
    assert lib.moegg_dispatch(e, at(0), at(1), at(2), at(3), at(0, 16), None, None) == INVALID   # overlap
    assert lib.moegg_dispatch(e, at(0), None, at(2), at(3), at(4), None, None) == INVALID
    assert lib.moegg_dispatch(e, at(0, 8), at(1), at(2), at(3), at(4), None, None) == MISALIGNED
    assert lib.moegg_combine(_exchange(dtype=1), at(0), at(1), None, None, at(4), None) == INVALID
    assert lib.moegg_combine(e, at(0), at(1), None, None, at(0, 64), None) == INVALID
    assert lib.moegg_combine(e, at(0), at(1), None, at(4, 16), at(4), None) == INVALID           # partial overlap
    assert lib.moegg_combine(e, None, at(1), None, None, at(4), None) == INVALID
    assert lib.moegg_combine_backward(e, at(0), at(1), at(2), at(3), at(4), None, at(5), None, None, None) == INVALID
    assert lib.moegg_combine_backward(e, at(0), at(1), at(2), at(3), None, None, at(5), None, at(6), None) == INVALID
    assert lib.moegg_combine_backward(e, at(0), at(1), at(2), at(3), at(5), None, at(5), None, at(6), None) == INVALID
    assert lib.moegg_unsort(at(0), at(1), at(2), -1, 5, None) == INVALID
    assert lib.moegg_unsort(None, at(1), at(2), 5, 5, None) == INVALID
    assert lib.moegg_unsort(None, None, None, 0, 5, None) == OK


def _linear(backward=False, prob=None, **args):
    p = dict(m=100, n=128, k=64, num_groups=1, act=0, dtype=3)
    p.update(prob or {})
    a = dict(x=at(0), w=at(1))
    a.update(dict(dy=at(2), dx=at(3), dw=at(4), db=at(5)) if backward else dict(y=at(6)))
    a.update(args)
    lib = mg._load()
    f = lib.moegg_linear_backward if backward else lib.moegg_linear
    return f(ctypes.byref(mg.moegg_linear_problem(**p)), ctypes.byref(mg.moegg_linear_args(**a)), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("prob,want", [
    (dict(m=-1), INVALID), (dict(m=1 << 31), NOT_SUPPORTED), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(n=132), NOT_SUPPORTED), (dict(k=60), NOT_SUPPORTED), (dict(n=(1 << 20) + 8), NOT_SUPPORTED),
    (dict(num_groups=0), INVALID), (dict(num_groups=1025), INVALID), (dict(num_groups=2), INVALID),  # no offsets
    (dict(act=5), INVALID), (dict(act=8), INVALID), (dict(act=1, n=96), INVALID), (dict(dtype=1), INVALID),
])
def test_linear_problem_refusals(back, prob, want):
    assert _linear(back, prob) == want, mg.moegg_last_error()


@pytest.mark.parametrize("back,prob,args,want", [
    (False, {}, dict(x=None), INVALID), (False, {}, dict(y=None), INVALID), (False, {}, dict(w=at(1, 8)), MISALIGNED),
    (False, {}, dict(bias=at(7, 2)), MISALIGNED), (False, {}, dict(y=at(0)), INVALID),
    (False, {}, dict(c=at(6)), INVALID), (False, {}, dict(residual=at(6, 16)), INVALID),
    (False, dict(dtype=5), dict(residual=at(6)), INVALID),           # in place, of another type
    (False, {}, dict(dy=at(2)), INVALID), (False, dict(m=0), dict(x=None, w=None, y=None), OK),
    (True, {}, dict(dy=None), INVALID), (True, {}, dict(dx=None, dw=None, db=None), INVALID),
    (True, dict(act=7), {}, INVALID),                                # no c
    (True, dict(act=7), dict(c=at(6)), INVALID),                     # no workspace
    (True, {}, dict(y=at(6)), INVALID), (True, {}, dict(dx=at(2)), INVALID), (True, {}, dict(w=None), INVALID),
    (True, {}, dict(x=None), INVALID), (True, {}, dict(dw=at(4, 4)), MISALIGNED),
])
def test_linear_pointer_refusals(back, prob, args, want):
    assert _linear(back, prob, **args) == want, mg.moegg_last_error()


@pytest.mark.parametrize("back,prob,args", [
    (False, {}, dict(y=at(1))), (False, {}, dict(c=at(1, 16))), (False, {}, dict(bias=at(6, 4))),
    (False, {}, dict(residual=at(7), c=at(7))), (False, {}, dict(offsets=at(6))),
    (True, {}, dict(dx=at(1))), (True, {}, dict(dx=at(4))), (True, {}, dict(dw=at(0))), (True, {}, dict(dw=at(2, 16))),
    (True, {}, dict(db=at(1))), (True, {}, dict(db=at(3, 4))), (True, dict(dtype=5), dict(dw=at(1))),
])
def test_linear_outputs_lie_apart(back, prob, args):
    """An output that shares memory with an operand or another output is refused."""
    size = mg._load().moegg_linear_backward_workspace(ctypes.byref(mg.moegg_linear_problem(100, 128, 64, 1, 0, 3)), 7)
    if back:
        args = dict(args, workspace=at(7), workspace_bytes=size)
    assert _linear(back, prob, **args) == INVALID and "overlap" in mg.moegg_last_error()


def test_launches_of_more_threads_than_32_bits_count_are_refused():
    big = (1 << 31) - 1024
    for prob in (dict(m=big, n=8, k=8), dict(m=big, n=8, k=512), dict(m=big, n=128, k=8),
                 dict(m=8, n=1 << 20, k=8, num_groups=1024)):
        for back in (False, True):
            assert _linear(back, prob, offsets=at(7, 512)) == NOT_SUPPORTED and "threads" in mg.moegg_last_error()
    assert mg._load().moegg_linear_workspace(ctypes.byref(mg.moegg_linear_problem(1 << 24, 64, 2048, 1, 0, 3))) >= 0
    assert _route(dict(num_tokens=1 << 28, top_k=2)) == NOT_SUPPORTED and "threads" in mg.moegg_last_error()
    assert _route(dict(num_tokens=1 << 26, num_experts=512, top_k=2)) == NOT_SUPPORTED
    lib = mg._load()
    for e in (_exchange(num_tokens=1 << 26, rows=1 << 26, top_k=1), _exchange(num_tokens=1 << 23, rows=1 << 10, width=8192)):
        assert lib.moegg_dispatch(e, at(0), at(1), at(2), at(3), at(4), None, None) == NOT_SUPPORTED
        assert lib.moegg_combine(e, at(0), at(1), None, None, at(4), None) == NOT_SUPPORTED


def test_linear_workspace_of_invalid_problems():
    lib = mg._load()
    assert lib.moegg_linear_workspace(ctypes.byref(mg.moegg_linear_problem(m=-1))) == -1
    assert lib.moegg_linear_backward_workspace(ctypes.byref(mg.moegg_linear_problem(m=8, n=4, k=8, num_groups=1, dtype=3)),
                                               7) == -1


# ---- refusals of the Python front -----------------------------------------------

def test_front_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        mg.route(x, 2)
    with pytest.raises(TypeError, match="dtype"):
        mg.route(x.double(), 2)
    with pytest.raises(TypeError, match="tensor expected"):
        mg.linear([1.0], x)
    with pytest.raises(ValueError, match="contiguous"):
        mg.linear(torch.zeros(64, 4, dtype=torch.bfloat16).t(), x)
    with pytest.raises(ValueError, match="shape"):
        mg.sort_tokens(torch.zeros(4, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="act"):
        mg.linear(x, x, act="geglu")
    with pytest.raises(ValueError, match="dtype"):
        mg.linear(x, x, dtype="e4m3")
    with pytest.raises(ValueError, match="need"):
        mg.linear_backward(x, x, x, need=("dy",))
    with pytest.raises(TypeError, match="SortPlan"):
        mg.layer._plan_pointers(None, 0)
    with pytest.raises(ValueError, match="score"):
        mg.layer._code(mg.SCORES, "relu", "score")


# ---- the reference itself -----------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_reference_route_gradient_against_differences(score, renormalise):
    gen = torch.Generator().manual_seed(11)
    t, e, k, scale = 5, 9, 3, 1.7
    x = torch.randn(t, e, generator=gen, dtype=torch.float64)
    x[1, 2] = -ref.INF
    x[2] = -ref.INF
    x[3, :7] = -ref.INF                                    # fewer experts than choices
    ids, _, _ = ref.route(x, k, score, renormalise=renormalise, scale=scale)
    assert (ids[2] == -1).all() and (ids[3] >= 0).sum() == 2
    g = torch.randn(t, k, generator=gen, dtype=torch.float64)
    d = ref.route_backward(x, ids, g, score, renormalise, scale)
    h = 1e-6
    for e0 in range(e):
        up, dn = x.clone(), x.clone()
        up[:, e0] += h
        dn[:, e0] -= h
        f = [(ref.weights_of(y, ids, _p(y, score), score, renormalise, scale) * g).sum(1) for y in (up, dn)]
        assert torch.allclose((f[0] - f[1]) / (2 * h), d[:, e0], atol=1e-8)


def _p(x, score):
    if score == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(1, keepdim=True)
    ex = torch.where(x == -ref.INF, 0.0, torch.exp(x - torch.where(top == -ref.INF, 0.0, top)))
    return ex / ex.sum(1, keepdim=True).clamp(min=1e-300)


def test_reference_exchange_gradients_against_differences():
    gen = torch.Generator().manual_seed(12)
    t, k, e, h = 4, 2, 3, 8
    ids = torch.tensor([[0, 2], [2, -1], [2, 0], [-1, -1]])
    rows = 4 * 8
    off, row_of, slot_of = ref.sort(ids, e, 4, rows)
    assert off.tolist() == [4, 4, 8] and row_of.tolist() == [[0, 4], [5, -1], [6, 1], [-1, -1]]
    assert slot_of[:8].tolist() == [0, 5, -1, -1, 1, 2, 4, -1]
    d = torch.randn(rows, h, generator=gen, dtype=torch.float64)
    w = torch.rand(t, k, generator=gen, dtype=torch.float64)
    dy = torch.randn(t, h, generator=gen, dtype=torch.float64)
    slot_w = torch.where(slot_of >= 0, w.reshape(-1)[slot_of.clamp(min=0)], 0.0)
    drows = ref.dispatch(dy, slot_of, k) * slot_w[:, None]
    eps = 1e-6
    for r, c in [(0, 0), (4, 3), (6, 7), (2, 1), (20, 0)]:
        up = d.clone()
        up[r, c] += eps
        diff = ((ref.combine(up, row_of, w)[0] - ref.combine(d, row_of, w)[0]) * dy).sum() / eps
        assert abs(diff - drows[r, c]) < 1e-6


@pytest.mark.parametrize("kind", ["none", "swiglu", "srelu", "gelu"])
def test_reference_linear_gradients_against_differences(kind):
    gen = torch.Generator().manual_seed(13)
    m, n, k = 7, 64, 16
    x = torch.randn(m, k, generator=gen, dtype=torch.float64)
    w = torch.randn(2, n, k, generator=gen, dtype=torch.float64)
    b = torch.randn(2, n, generator=gen, dtype=torch.float64)
    off = torch.tensor([3, 7])
    y, z, _ = ref.linear(x, w, b, kind, None, off)
    dy = torch.randn_like(y)
    got = ref.linear_backward(dy, x, w, z, kind, off)
    eps = 1e-6

    def diff(**kw):
        a = dict(x=x, w=w, bias=b, kind=kind, offsets=off)
        a.update(kw)
        return ((ref.linear(**a)[0] - y) * dy).sum() / eps
    for name, t, grad in (("x", x, "dx"), ("w", w, "dw"), ("bias", b, "db")):
        for i in (0, 5, t.numel() - 1):
            up = t.clone().reshape(-1)
            up[i] += eps
            want = got[grad][0].reshape(-1)[i]
            assert abs(diff(**{name: up.reshape(t.shape)}) - want) < 1e-3 * (1 + abs(want))
