"""Sizes of tensors that the C structs' 32-bit fields do not hold are refused
by the front (a field cuts a longer number without a word, and the call would
work on the tensor's first columns).  Tensors without memory, no GPU."""
import os

import pytest

torch = pytest.importorskip("torch")

import moe_grouped_block_amd as mg  # noqa: E402

BIG = 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


@pytest.fixture()
def front(monkeypatch):
    """The front with its checks of place taken for passed, and no call behind it."""
    def enqueued(*_):
        raise AssertionError("the call went through")
    layer = mg.layer
    monkeypatch.setattr(layer, "_lead", lambda t, *_: 0)
    monkeypatch.setattr(layer, "_want", lambda *_: 0)
    monkeypatch.setattr(layer, "_on", enqueued)


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def plan(t, k, rows, experts=4):
    i32 = torch.int32
    return mg.SortPlan(experts, 1, meta(experts, dtype=i32), meta(t, k, dtype=i32), meta(rows, dtype=i32))


@pytest.mark.parametrize("call", [
    lambda: mg.route(meta(1, BIG + 64), 2),
    lambda: mg.route_backward(meta(1, BIG + 64), meta(1, 2, dtype=torch.int32), meta(1, 2, dtype=torch.float32)),
    lambda: mg.route_backward(meta(1, 64), meta(1, BIG + 2, dtype=torch.int32), meta(1, BIG + 2, dtype=torch.float32)),
    lambda: mg.sort_tokens(meta(1, BIG + 2, dtype=torch.int32), 4),
    lambda: mg.dispatch(meta(1, BIG + 8), plan(1, 2, 2)),
    lambda: mg.dispatch(meta(1, 8), plan(1, BIG + 2, 2)),
    lambda: mg.combine(meta(2, BIG + 8), plan(1, 2, 2)),
    lambda: mg.combine(meta(2, 8), plan(1, BIG + 2, 2)),
    lambda: mg.combine_backward(meta(1, BIG + 8), plan(1, 2, 2)),
    lambda: mg.dispatch_backward(meta(2, BIG + 8), plan(1, 2, 2)),
    lambda: mg.linear(meta(1, BIG + 8), meta(8, BIG + 8)),
    lambda: mg.linear(meta(1, 8), meta(BIG + 8, 8)),
    lambda: mg.linear(meta(1, 8), meta(BIG + 1, 8, 8), offsets=meta(BIG + 1, dtype=torch.int32)),
    lambda: mg.linear_backward(meta(1, BIG + 8), meta(1, 8), meta(BIG + 8, 8)),
])
def test_sizes_past_32_bits_are_refused(front, call):
    with pytest.raises(ValueError, match="2\\^31"):
        call()


def test_sizes_in_range_pass(front):
    for call in (lambda: mg.route(meta(1, 64), 2), lambda: mg.linear(meta(1, 8), meta(8, 8)),
                 lambda: mg.dispatch(meta(1, 8), plan(1, 2, 2))):
        with pytest.raises(AssertionError, match="went through"):
            call()
