"""linear_backward of the C ABI without rows (no GPU: nothing is enqueued)."""
import ctypes
import os

import pytest

pytest.importorskip("torch")
import moe_grouped_block_amd as mg  # noqa: E402

OK, INVALID = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


@pytest.mark.parametrize("act", [0, 1, 7])
def test_no_gradient_is_required_without_rows(act):
    """dx of no rows has no memory: NULL, as an empty tensor's address is."""
    args = ctypes.byref(mg.moegg_linear_args())
    lib = mg._load()
    assert lib.moegg_linear_backward(ctypes.byref(mg.moegg_linear_problem(0, 64, 64, 1, act, 3)), args, None) == OK
    assert lib.moegg_linear_backward(ctypes.byref(mg.moegg_linear_problem(1, 64, 64, 1, act, 3)), args, None) == INVALID
