"""moegg_run with more rows than padded_offsets names (the capacity that
sort_tokens works with): the rows in use get the same bits as without the rest,
the rest is neither read (it holds NaN) nor written, for every kind of output."""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
from moe_grouped_block_amd import plumbing as pl  # noqa: E402

MARK = 0xA5
L = 5
FORCED, ROUTED = dict(force_counts=[130, 0, 1, 256, 300]), dict(routing=("topk", 220, 2))
# (the backwards with 64 columns: one wave adds to a row's dprob, so that its order is the same)
CASES = {
    "gating_bf16_d": ("quant_gating_l4", dict(FORCED, K=512, N=320)),
    "swiglu_e4m3": ("fc1_swiglu_l8", dict(FORCED, K=512, N=320)),
    "srelu_fp4_c": ("srelu_tanh_fp4_l32", dict(FORCED, K=1024, N=320, c="bf16")),
    "geglu_e5m2": ("fc1_geglu_e5m2_l8", dict(FORCED, K=768, N=320)),
    "dswiglu_bf16": ("dswiglu_bf16_l64", dict(ROUTED, K=512, N=64)),
    "dswiglu_e4m3": ("dswiglu_mxfp8_l64", dict(ROUTED, K=640, N=64)),
    "dsrelu_e4m3": ("dsrelu_mxfp8_l32", dict(ROUTED, K=512, N=64)),
    "dgeglu_e4m3": ("dgeglu_mxfp8_l64", dict(ROUTED, K=384, N=64)),
}


def longer(arrays, extra):
    """Every row tensor with `extra` rows of NaN behind it."""
    out = dict(arrays)
    for name, nan in (("a", {np.uint8: 0x7F, np.uint16: 0x7FC0}), ("sfa", {np.uint8: 0xFF}), ("prob", {np.float32: np.nan}),
                      ("c_in", {np.uint16: 0x7FC0})):
        if name in out:
            v = out[name]
            out[name] = np.concatenate([v, np.full((extra, *v.shape[1:]), nan[v.dtype.type], v.dtype)])
    return out


def run(problem, arrays, layout):
    p = dict(problem, sf_layout=layout)
    dev = pl.to_device(arrays, sf_layout=layout, k=p["k"])
    outs = pl.empty_outputs(p, fill=MARK)
    mg.run(p, {**pl.inputs_for(p, dev), **outs})
    torch.cuda.synchronize()
    return pl.to_host(outs)


@pytest.mark.parametrize("extra", [128, 1152])
@pytest.mark.parametrize("name,layout", [(n, lay) for n in CASES for lay in ("row_major", "kplanes")
                                         if lay == "row_major" or n != "dswiglu_bf16"])      # (BF16 has no scales)
def test_rows_behind_the_last_group(name, layout, extra):
    base, over = CASES[name]
    case = synth.make_case(base, seed=9100 + extra, name=name, L=L, **over)
    p, used = case.problem, case.problem["valid_m"]
    print(f"\n[gpu-case] {name} rows in use {used} of {used + extra} {layout}", flush=True)
    want = run(p, case.arrays, layout)
    got = run(dict(p, valid_m=used + extra), longer(case.arrays, extra), layout)
    assert set(got) == set(want)
    for key, g in got.items():
        w = want[key]
        if key == "amax":
            assert np.array_equal(g, w)
        elif key == "sfd_col":                       # (N_out, rows / 32)
            assert np.array_equal(g[:, :used // 32], w) and (g[:, used // 32:] == MARK).all()
        else:
            assert np.array_equal(g[:used], w, equal_nan=g.dtype == np.float32), key
            rest = g[used:]
            assert (rest == 0).all() if key == "dprob" else (rest.view(np.uint8) == MARK).all(), key


@pytest.mark.parametrize("name", list(CASES))
def test_no_rows_in_use(name):
    """Offsets that are all zero: nothing but amax (zero) is written."""
    base, over = CASES[name]
    case = synth.make_case(base, seed=9200, name=name, L=L, **over)
    arrays = longer(case.arrays, 128)
    arrays["padded_offsets"] = np.zeros_like(arrays["padded_offsets"])
    print(f"\n[gpu-case] {name} no rows in use", flush=True)
    got = run(dict(case.problem, valid_m=case.problem["valid_m"] + 128), arrays, "row_major")
    for key, g in got.items():
        assert (g == 0).all() if key in ("amax", "dprob") else (g.view(np.uint8) == MARK).all(), key


def test_check_offsets_of_a_sorted_plan():
    """moegg_check_offsets asks for the pages' own rule, valid_m == the last
    offset: a plan passes with its rows in use as valid_m, and not with its
    capacity, which moegg_run takes too."""
    t, e, k = 200, 6, 2
    ids = torch.randint(0, e, (t, k), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    plan = mg.sort_tokens(ids, e)
    used = int(plan.padded_offsets[-1])
    assert used < plan.rows
    p = dict(num_groups=e, n=64, k=128, ab_dtype="e4m3", d_dtype="bf16", act="none")
    at = plan.padded_offsets.data_ptr()
    assert mg.moegg_check_offsets(mg.make_problem(dict(p, valid_m=used)), at, None) == 0
    assert mg.moegg_check_offsets(mg.make_problem(dict(p, valid_m=plan.rows)), at, None) == 1
    assert "valid_m" in mg.moegg_last_error()
    assert mg.moegg_check_offsets(mg.make_problem(dict(p, valid_m=used - 128)), at, None) == 1
