"""The binding by itself needs no torch: the package imports, loads the
library and checks calls without it; only the layer operators bring it in."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

import moe_grouped_block_amd as mg  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(mg.lib_path):
        from moe_grouped_block_amd import build
        build.build()


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_the_binding_without_torch():
    out = python("""
import sys
sys.modules["torch"] = None                       # every import of torch fails
import moe_grouped_block_amd as mg
import moe_grouped_block_amd.build
from moe_grouped_block_amd import *
assert moegg_abi_version() == ABI_VERSION
p = dict(num_groups=1, valid_m=128, n=64, k=128, ab_dtype="e4m3", d_dtype="bf16", act="none")
at = 0x7F0000000000
t = {n: at + (i << 32) for i, n in enumerate(("a", "b", "sfa", "sfb", "padded_offsets", "alpha", "prob", "d", "amax"))}
mg.check(p, t)                                    # integer addresses: nothing is touched
for name in ("route", "layer", "SortPlan"):
    try:
        getattr(mg, name)
    except ImportError as e:
        assert "torch" in str(e)
    else:
        raise SystemExit(name + " without torch")
try:
    mg.no_such_name
except AttributeError as e:
    assert "no_such_name" in str(e)
print("fine")
""")
    assert out.strip() == "fine"


def test_the_import_does_not_bring_torch():
    assert python("import sys, moe_grouped_block_amd as mg; mg.moegg_abi_version(); print('torch' in sys.modules)").strip() == "False"


def test_every_public_name_is_there():
    pytest.importorskip("torch")
    for name in mg.__all__:
        assert getattr(mg, name) is not None
    assert set(mg.layer.__all__) <= set(mg.__all__) <= set(dir(mg))
    assert mg.route is mg.layer.route
    out = python("from moe_grouped_block_amd import *\nfrom moe_grouped_block_amd import linear as l\nprint(l is linear, route.__name__)")
    assert out.split() == ["True", "route"]
