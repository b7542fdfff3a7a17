"""What linear's ``save_c`` takes: truth values, and the names and torch types
that stand for a type of c; another type is refused and no other c is kept in
its place.  Tensors without memory, no GPU."""
import os

import pytest

torch = pytest.importorskip("torch")

import moe_grouped_block_amd as mg  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()



@pytest.fixture()
def calls(monkeypatch):
    """The front with its checks of place taken for passed and the library's calls noted."""
    made = []
    lib = mg._load()

    class Lib:
        moegg_linear_workspace = staticmethod(lib.moegg_linear_workspace)
        moegg_linear_saving_workspace = staticmethod(lib.moegg_linear_saving_workspace)

        @staticmethod
        def moegg_linear(p, a, stream):
            made.append(("bf16", bool(a.c)))
            return 0

        @staticmethod
        def moegg_linear_saving(p, a, keep, stream):
            made.append((keep.c_dtype, bool(a.c)))
            return 0
    monkeypatch.setattr(mg.layer, "_lead", lambda t, *_: 0)
    monkeypatch.setattr(mg.layer, "_want", lambda *_: 0)
    monkeypatch.setattr(mg.layer, "_on", lambda *_: (0, None))
    monkeypatch.setattr(mg, "_load", lambda: Lib)
    return made


def linear(save_c):
    # (tensors of the host: their c has an address)
    return mg.linear(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16), save_c=save_c)


@pytest.mark.parametrize("name", [torch.float8_e4m3fn, torch.float8_e5m2, torch.float32, torch.float16, torch.uint8, "f32", "e2m1x2",
                                  "float8_e4m3fn"])
def test_other_types_are_refused(calls, name):
    with pytest.raises(ValueError, match="save_c"):
        linear(name)
    assert not calls


@pytest.mark.parametrize("save_c,kept", [(False, ("bf16", False)), (None, ("bf16", False)), (True, ("bf16", True)),
                                         (torch.bfloat16, ("bf16", True)), ("bf16", ("bf16", True)), ("e4m3", (1, True)),
                                         ("e5m2", (4, True))])
def test_what_is_kept(calls, save_c, kept):
    got = linear(save_c)
    assert calls == [kept]
    if kept == ("bf16", False):
        assert got.shape == (2, 64)
    elif kept[0] == "bf16":
        assert got[1].dtype is torch.bfloat16 and got[1].shape == (2, 64)
    else:
        codes, scales = got[1]
        assert codes.dtype is torch.uint8 and codes.shape == (2, 64) and scales.shape == (2, 2)
