"""A library built before a function of these bindings existed says that it
has to be rebuilt (its version number counts the structs' layouts, which new
functions leave alone)."""
import ctypes
import subprocess

import pytest

import moe_grouped_block_amd as mg


@pytest.mark.parametrize("version,functions", [
    (mg.ABI_VERSION, ("moegg_check", "moegg_run", "moegg_check_offsets", "moegg_n_out", "moegg_status_string",
                      "moegg_last_error", "moegg_set_grid_limit", "moegg_sf_to_kplanes")),   # without the layer operators
    (mg.ABI_VERSION, ()),
    (mg.ABI_VERSION - 1, ("moegg_check",)),
])
def test_a_library_built_before(tmp_path, monkeypatch, version, functions):
    src, lib = tmp_path / "old.c", tmp_path / "libold.so"
    src.write_text(f"int moegg_abi_version(void) {{ return {version}; }}\n" +
                   "".join(f"int {f}(void) {{ return 0; }}\n" for f in functions))
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    monkeypatch.setattr(mg, "lib_path", str(lib))
    monkeypatch.setattr(mg, "_lib", None)
    with pytest.raises(RuntimeError, match="rebuild") as e:
        mg.moegg_abi_version()
    assert str(lib) in str(e.value)
    assert mg._lib is None


def test_no_library_of_this_project(tmp_path, monkeypatch):
    src, lib = tmp_path / "none.c", tmp_path / "libnone.so"
    src.write_text("int something_else(void) { return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    ctypes.CDLL(str(lib))
    monkeypatch.setattr(mg, "lib_path", str(lib))
    monkeypatch.setattr(mg, "_lib", None)
    with pytest.raises(RuntimeError, match="rebuild"):
        mg.moegg_abi_version()
