"""The layer operators together, as an MoE block uses them: forward and
backward against float64 autograd, MX rows into the grouped product, captured
into graphs, and on several streams at once."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402
import oracle  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu


class Block:
    """Router, experts (gated first product, second product), a shared expert
    whose result is the residual of the combination; BF16."""

    def __init__(self, t=150, h=256, f=128, e=8, k=3, m_aligned=1, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def bf(*s, scale=1.0):
            return (torch.randn(*s, generator=gen) * scale).to(torch.bfloat16)
        self.e, self.k, self.ma = e, k, m_aligned
        self.x, self.dy = bf(t, h), bf(t, h)
        self.wr, self.br = bf(e, h, scale=1 / math.sqrt(h)), torch.randn(e, generator=gen) * 0.1
        self.w1, self.b1 = bf(e, 2 * f, h, scale=1 / math.sqrt(h)), torch.randn(e, 2 * f, generator=gen) * 0.1
        self.w2 = bf(e, h, f, scale=1 / math.sqrt(f))
        self.s1, self.s2 = bf(f, h, scale=1 / math.sqrt(h)), bf(h, f, scale=1 / math.sqrt(f))
        self.bs = torch.randn(f, generator=gen) * 0.1

    def to(self, dev):
        b = Block.__new__(Block)
        b.__dict__ = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in self.__dict__.items()}
        return b

    def step(self, stream=None):
        """One training step's forward and backward: y and every gradient."""
        s = dict(stream=stream)
        logits = mg.linear(self.x, self.wr, bias=self.br, dtype="f32", **s)
        ids, w = mg.route(logits, self.k, **s)
        plan = mg.sort_tokens(ids, self.e, m_aligned=self.ma, **s)
        a = mg.dispatch(self.x, plan, **s)
        h1, c1 = mg.linear(a, self.w1, bias=self.b1, act="swiglu", offsets=plan.padded_offsets, save_c=True, **s)
        d = mg.linear(h1, self.w2, offsets=plan.padded_offsets, **s)
        hs, cs = mg.linear(self.x, self.s1, bias=self.bs, act="gelu", save_c=True, **s)
        shared = mg.linear(hs, self.s2, residual=self.x, **s)
        y = mg.combine(d, plan, weights=w, residual=shared, **s)
        dd, dw = mg.combine_backward(self.dy, plan, rows=d, weights=w, **s)
        dh1, dw2, _ = mg.linear_backward(dd, h1, self.w2, offsets=plan.padded_offsets, need=("dx", "dw"), **s)
        da, dw1, db1 = mg.linear_backward(dh1, a, self.w1, c=c1, act="swiglu", offsets=plan.padded_offsets, **s)
        dx_routed = mg.dispatch_backward(da, plan, **s)
        dlogits = mg.route_backward(logits, ids, dw, **s).to(torch.bfloat16) if stream is None else None
        dhs, ds2, _ = mg.linear_backward(self.dy, hs, self.s2, need=("dx", "dw"), **s)
        dx_shared, ds1, dbs = mg.linear_backward(dhs, self.x, self.s1, c=cs, act="gelu", **s)
        out = dict(y=y, ids=ids, dx_routed=dx_routed, dx_shared=dx_shared, dw1=dw1, db1=db1, dw2=dw2, ds1=ds1, ds2=ds2,
                   dbs=dbs, dweights=dw)
        if dlogits is not None:
            out["dx_router"], out["dwr"], out["dbr"] = mg.linear_backward(dlogits, self.x, self.wr)
        return out

    def reference(self, ids):
        """The same in float64 through autograd, for the choice `ids`."""
        p = {n: getattr(self, n).double().clone().requires_grad_(True)
             for n in ("x", "wr", "br", "w1", "b1", "w2", "s1", "bs", "s2")}
        xs = {n: p["x"].detach().clone().requires_grad_(True) for n in ("router", "routed", "shared")}
        logits = xs["router"] @ p["wr"].t() + p["br"]
        soft = torch.softmax(logits.gather(1, ids), 1)
        soft.retain_grad()
        y = self.x.double()
        for g in range(self.e):
            tok, j = (ids == g).nonzero(as_tuple=True)
            z = xs["routed"][tok] @ p["w1"][g].t() + p["b1"][g]
            o = ref.act(z, "swiglu") @ p["w2"][g].t() * soft[tok, j][:, None]
            y = y.index_add(0, tok, o)
        hs = ref.act(xs["shared"] @ p["s1"].t() + p["bs"], "gelu")
        y = y + hs @ p["s2"].t()
        y.backward(self.dy.double())
        return dict(y=y.detach(), dx_routed=xs["routed"].grad, dx_shared=xs["shared"].grad, dx_router=xs["router"].grad,
                    dw1=p["w1"].grad, db1=p["b1"].grad, dw2=p["w2"].grad, ds1=p["s1"].grad, ds2=p["s2"].grad,
                    dbs=p["bs"].grad, dwr=p["wr"].grad, dbr=p["br"].grad, dweights=soft.grad)


@pytest.mark.parametrize("kw", [dict(), dict(t=1), dict(t=2, k=1, e=64), dict(t=77, m_aligned=128), dict(t=500, f=320, h=520)])
def test_block_forward_and_backward(kw):
    """Each output passes at most eight bf16 roundings (2^-8 each at most, of
    values that add up over the sums): as vectors they agree to a few 2^-8."""
    b = Block(**kw)
    print(f"[gpu-case] block {kw}", flush=True)
    got = b.to("cuda").step()
    want = b.reference(got["ids"].cpu().long())
    for name, r in want.items():
        g = got[name].cpu().double()
        assert g.shape == r.shape
        scale = r.norm()
        if kw.get("k") == 1 and name in ("dx_router", "dwr", "dbr"):
            # one weight is always 1: no gradient but the cancellation's rounding
            assert g.abs().max() < 1e-4
            continue
        assert (g - r).norm() <= 4 * ref.BF16 * scale, (name, float((g - r).norm() / scale))


def _tensors(out):
    return {k: v for k, v in out.items() if v is not None}


def test_block_in_a_graph():
    """Forward and backward captured once and replayed on new inputs, with
    eager work between the replays; every replay equals the eager result."""
    b = Block(t=100, m_aligned=1).to("cuda")
    for _ in range(2):
        b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for rep in range(4):
        new = Block(t=100, m_aligned=1, seed=rep + 10)
        b.x.copy_(new.x)
        b.dy.copy_(new.dy)
        for v in _tensors(out).values():
            v.view(torch.uint8).fill_(0x5A + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = b.step()
        torch.cuda.synchronize()
        for name, v in _tensors(out).items():
            assert torch.equal(v, eager[name]), (rep, name)
    del graph


def test_two_graphs_replayed_side_by_side():
    """Graphs captured with workspaces of their own, replayed on two streams at once."""
    bs = [Block(t=700, m_aligned=1, seed=i).to("cuda") for i in (1, 2)]
    want = [b.step() for b in bs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in bs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for name in w:
                assert torch.equal(o[name], w[name]), name
    del graphs


def test_streams_given_by_argument():
    """Two blocks on two streams passed as arguments, while the current stream is another."""
    bs = [Block(t=400, m_aligned=128, seed=i).to("cuda") for i in (3, 4)]
    want = [b.step() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(3):
        got = [b.step(stream=s) for b, s in zip(bs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for name in g:
                assert torch.equal(g[name], w[name]), name
    raw = bs[0].step(stream=streams[0].cuda_stream)
    streams[0].synchronize()
    for name in raw:
        assert torch.equal(raw[name], want[0][name])


def test_results_do_not_depend_on_the_run():
    b = Block(t=2000, e=16, k=4).to("cuda")
    first = b.step()
    for _ in range(5):
        again = b.step()
        for name in first:
            assert torch.equal(first[name], again[name]), name


@pytest.mark.parametrize("layout", ["row_major", "kplanes"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1x2"])
def test_mx_rows_into_the_grouped_product(fmt, layout):
    """route -> sort -> dispatch writes moegg_run's A, SFA, padded_offsets and
    prob; moegg_run takes the capacity as valid_m, gives the oracle's result on
    the rows in use, and leaves the rows behind the last expert; combine adds
    the gated rows."""
    t, e, k, n, kk = 210, 6, 2, 96, 512
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(t, kk, generator=gen).to(torch.bfloat16)
    w = torch.randn(e, n, kk, generator=gen) / math.sqrt(kk)
    b, sfb = synth.mx_quantize(w.numpy(), fmt)
    logits = torch.randn(t, e, generator=gen)
    logits[:, 2] = -math.inf                              # an expert without rows
    print(f"[gpu-case] MX rows {fmt} {layout}", flush=True)
    ids, wt = mg.route(logits.cuda(), k)
    plan = mg.sort_tokens(ids, e, weights=wt)
    a, sfa = mg.dispatch(x.cuda(), plan, dtype=fmt, sf_layout=layout)
    p = dict(num_groups=e, valid_m=plan.rows, n=n, k=kk, ab_dtype=fmt, d_dtype="bf16", act="none", sf_layout=layout)
    used = int(plan.padded_offsets[-1])
    assert used < plan.rows
    d = torch.full((plan.rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    amax = torch.empty(e, device="cuda")
    sfb_d = torch.from_numpy(sfb).cuda()
    if layout == "kplanes":
        planes = torch.empty(sfb.size, dtype=torch.uint8, device="cuda")
        mg.sf_to_kplanes(sfb_d, planes, e * n, kk)
        sfb_d = planes
    mg.run(p, dict(a=a, sfa=sfa, b=torch.from_numpy(b).cuda(), sfb=sfb_d, padded_offsets=plan.padded_offsets,
                   alpha=torch.ones(e, device="cuda"), prob=plan.prob, d=d, amax=amax))
    assert (d[used:] == 7.0).all()
    sfa_h = sfa.cpu().numpy()
    if layout == "kplanes":
        sfa_h = sfa_h.transpose(1, 0, 2).reshape(plan.rows, -1)
    host = dict(a=a.cpu().numpy()[:used], sfa=np.ascontiguousarray(sfa_h[:used]), b=b, sfb=sfb,
                padded_offsets=plan.padded_offsets.cpu().numpy(), alpha=np.ones(e, np.float32),
                prob=plan.prob.cpu().numpy()[:used])
    r = oracle.grouped_gemm({**p, "valid_m": used, "m_aligned": 128, "sf_layout": "row_major"}, host)
    got, want = d[:used].float().cpu().numpy(), np.asarray(r["d"], np.float64)
    assert np.abs(got - want).max() <= 1e-2 * np.abs(want).max()
    y = mg.combine(d, plan)
    s, mag = ref.combine(d.cpu(), plan.row_of.cpu().long())
    assert ((y.cpu().double() - s).abs() <= ref.BF16 * s.abs() + 8 * ref.F32 * mag).all()


def test_tensors_are_checked():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    plan = mg.sort_tokens(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    for call, err in [
        (lambda: mg.linear(x, w[:, :32].contiguous()), ValueError), (lambda: mg.linear(x, w.cpu()), ValueError),
        (lambda: mg.linear(x, w, bias=torch.zeros(8, device="cuda", dtype=torch.bfloat16)), TypeError),
        (lambda: mg.linear(x, w, residual=x), ValueError), (lambda: mg.linear(x, w, act="swiglu"), mg.MoeggError),
        (lambda: mg.linear(x[:, 1:57], w), ValueError), (lambda: mg.linear(x, w, out=x), ValueError),
        (lambda: mg.linear_backward(x[:, :8].contiguous(), x, w, act="gelu"), ValueError),
        (lambda: mg.route(x, 33), mg.MoeggError), (lambda: mg.route(x, 0), mg.MoeggError),
        (lambda: mg.route(x, -1), ValueError),
        (lambda: mg.dispatch(x[:3], plan), ValueError), (lambda: mg.dispatch(x, plan, dtype="e4m3"), mg.MoeggError),
        (lambda: mg.dispatch(x, plan, out=x), ValueError), (lambda: mg.combine(x, plan), ValueError),
        (lambda: mg.dispatch(x, plan, dtype="f32"), ValueError),
        (lambda: mg.sort_tokens(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), 3), TypeError),
        (lambda: mg.sort_tokens(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 0), mg.MoeggError),
        (lambda: mg.unsort(torch.zeros(5, device="cuda"), plan), ValueError),
    ]:
        with pytest.raises(err):
            call()
