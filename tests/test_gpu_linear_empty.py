"""linear_backward without rows: whichever gradients are asked for."""
import itertools

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")

pytestmark = pytest.mark.gpu

NEEDS = [c for r in (1, 2, 3) for c in itertools.combinations(("dx", "dw", "db"), r)]


@pytest.mark.parametrize("need", NEEDS)
@pytest.mark.parametrize("groups", [0, 3])
@pytest.mark.parametrize("act", ["none", "swiglu", "gelu"])
def test_backward_without_rows(need, groups, act):
    n, k = 64, 72
    w = torch.randn(*((groups, n, k) if groups else (n, k)), device="cuda").to(torch.bfloat16)
    x = torch.empty(0, k, device="cuda", dtype=torch.bfloat16)
    dy = torch.empty(0, n // 2 if act == "swiglu" else n, device="cuda", dtype=torch.bfloat16)
    c = torch.empty(0, n, device="cuda", dtype=torch.bfloat16) if act != "none" else None
    off = torch.zeros(groups, dtype=torch.int32, device="cuda") if groups else None
    print(f"[gpu-case] linear backward m=0 {act} groups={groups} {need}", flush=True)
    dx, dw, db = mg.linear_backward(dy, x, w, c=c, act=act, offsets=off, need=need)
    assert (dx is None) == ("dx" not in need) and (dw is None) == ("dw" not in need) and (db is None) == ("db" not in need)
    if dx is not None:
        assert dx.shape == (0, k)
    for g, shape in ((dw, w.shape), (db, w.shape[:-1])):
        if g is not None:
            assert g.shape == shape and (g == 0).all()
