"""The norm, the router with groups and activations kept in 8 bits together,
as a training step of an MoE block with its norm uses them: forward and
backward against float64, in graphs, on streams and inside autograd."""
import math

import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref  # noqa: E402
import more_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Block:
    """Residual and norm, a router that chooses groups, experts of two products.
    What the backward reads of the products' inputs and of c is kept in 8 bits."""

    def __init__(self, t=150, h=256, f=128, e=16, k=3, groups=4, top_groups=2, best=2, layout="row_major", seed=0):
        gen = torch.Generator().manual_seed(seed)

        def bf(*s, scale=1.0):
            return (torch.randn(*s, generator=gen) * scale).to(BF)
        self.e, self.k, self.layout = e, k, layout
        self.how = dict(score="sigmoid", num_groups=groups, top_groups=top_groups, group_best=best)
        self.x, self.stream_in, self.dout = bf(t, h), bf(t, h, scale=3.0), bf(t, h)
        self.norm = torch.rand(h, generator=gen) + 0.5
        self.wr, self.balance = bf(e, h, scale=1 / math.sqrt(h)), torch.randn(e, generator=gen) * 0.05
        self.w1, self.b1 = bf(e, 2 * f, h, scale=1 / math.sqrt(h)), torch.randn(e, 2 * f, generator=gen) * 0.1
        self.w2 = bf(e, h, f, scale=1 / math.sqrt(f))

    def to(self, dev):
        b = Block.__new__(Block)
        b.__dict__ = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in self.__dict__.items()}
        return b

    def step(self, stream=None):
        s = dict(stream=stream)
        lay = dict(sf_layout=self.layout)
        y, y8, h = mg.rms_norm(self.x, self.norm, residual=self.stream_in, copy="e4m3", **lay, **s)
        logits = mg.linear(y, self.wr, dtype="f32", **s)
        ids, w = mg.route(logits, self.k, bias=self.balance, **self.how, **s)
        plan = mg.sort_tokens(ids, self.e, m_aligned=1, **s)
        ends = dict(offsets=plan.padded_offsets)
        a, a8 = mg.dispatch(y, plan, **s), mg.dispatch(y, plan, dtype="e4m3", **lay, **s)
        h1, c8 = mg.linear(a, self.w1, bias=self.b1, act="swiglu", save_c="e5m2", **ends, **s)
        h8 = mg.quantise(h1, **s)
        d = mg.linear(h1, self.w2, **ends, **s)
        out = mg.combine(d, plan, weights=w, residual=h, **s)
        dd, dw = mg.combine_backward(self.dout, plan, rows=d, weights=w, **s)
        dh1, dw2, _ = mg.linear_backward(dd, h8, self.w2, x_dtype="e4m3", need=("dx", "dw"), **ends, **s)
        da, dw1, db1 = mg.linear_backward(dh1, a8, self.w1, c=c8, act="swiglu", x_dtype="e4m3", c_dtype="e5m2", **ends, **lay, **s)
        dy = mg.dispatch_backward(da, plan, **s)
        got = dict(out=out, h=h, y=y, ids=ids, w=w, dweights=dw, dw1=dw1, db1=db1, dw2=dw2, dy_routed=dy)
        kept = dict(y8=y8, a8=a8, h8=h8, c8=c8, logits=logits, row_of=plan.row_of, offsets=plan.padded_offsets)
        if stream is None:
            dlogits = mg.route_backward(logits, ids, dw, score="sigmoid").to(BF)
            dyr, got["dwr"], _ = mg.linear_backward(dlogits, y8, self.wr, x_dtype="e4m3", need=("dx", "dw"), **lay)
            dy = dy + dyr
            got["dlogits"] = dlogits
        got["dx"], got["dnorm"] = mg.rms_norm_backward(dy, h, self.norm, dh=self.dout, **s)
        return got, kept

    def reference(self, ids, kept):
        """The same in float64, for the choice `ids` and the activations that were kept, as they were kept."""
        t = self.x.shape[0]
        h = self.x.double() + self.stream_in.double()
        y = ref.rms_norm(h, self.norm, 1e-6)
        logits = y @ self.wr.double().t()
        p = torch.sigmoid(logits)
        w = layer_ref.weights_of(logits, ids, p, "sigmoid", True, 1.0)
        row_of, ends = kept["row_of"].cpu().long(), kept["offsets"].cpu()
        used = int(ends[-1])
        slot_of = torch.full((used,), -1, dtype=torch.int64)
        slot_of[row_of.reshape(-1)[row_of.reshape(-1) >= 0]] = (row_of.reshape(-1) >= 0).nonzero()[:, 0]
        token = slot_of // self.k

        def value(pair, fmt, layout="row_major"):
            return ref.decode(pair[0].cpu(), ref.rowmajor(pair[1].cpu(), layout), fmt)[:used]
        a8, c8, h8 = value(kept["a8"], "e4m3", self.layout), value(kept["c8"], "e5m2"), value(kept["h8"], "e4m3")
        y8 = ref.decode(kept["y8"][0].cpu(), ref.rowmajor(kept["y8"][1].cpu(), self.layout), "e4m3")
        h1, _, _ = layer_ref.linear(y[token], self.w1, self.b1, "swiglu", None, ends)
        d, _, _ = layer_ref.linear(h1, self.w2, None, "none", None, ends)
        out, _ = layer_ref.combine(d, row_of, w, h)
        dout, ws = self.dout.double(), w.reshape(-1)[slot_of]
        dweights = torch.zeros(t * self.k, dtype=torch.float64)
        dweights[slot_of] = (dout[token] * d).sum(1)
        dweights = dweights.reshape(t, self.k)
        b2 = layer_ref.linear_backward(dout[token] * ws[:, None], h8, self.w2, None, "none", ends)
        b1 = layer_ref.linear_backward(b2["dx"][0], a8, self.w1, c8, "swiglu", ends)
        dy = torch.zeros_like(h).index_add(0, token, b1["dx"][0])
        dlogits = layer_ref.route_backward(logits, ids, dweights, "sigmoid")
        dx, _, dnorm, _ = ref.rms_norm_backward(dy + dlogits @ self.wr.double(), h, self.norm, 1e-6, dout)
        return dict(out=out, h=h, y=y, w=w, dweights=dweights, dw1=b1["dw"][0], db1=b1["db"][0], dw2=b2["dw"][0], dy_routed=dy,
                    dlogits=dlogits, dwr=dlogits.t() @ y8, dx=dx, dnorm=dnorm)


@pytest.mark.parametrize("kw", [dict(), dict(t=1), dict(t=77, layout="kplanes"), dict(t=500, f=160, h=640, e=24, groups=3, best=1),
                                dict(t=300, e=8, k=2, groups=8, top_groups=5, best=1)])
def test_forward_and_backward(kw):
    """Each output passes at most eight bf16 roundings (2^-8 each at most, of
    values that add up over the sums): as vectors they agree to a few 2^-8."""
    b = Block(**kw)
    print(f"[gpu-case] block with norm {kw}", flush=True)
    got, kept = b.to("cuda").step()
    ids = got["ids"].cpu().long()
    assert torch.equal(ids, ref.route_grouped(kept["logits"].cpu(), b.k, b.how["num_groups"], b.how["top_groups"],
                                              b.how["group_best"], "sigmoid", b.balance))
    want = b.reference(ids, kept)
    assert set(want) == set(got) - {"ids"}
    for name, r in want.items():
        g = got[name].cpu().double()
        assert g.shape == r.shape
        assert (g - r).norm() <= 4 * ref.BF16 * r.norm(), (name, float((g - r).norm() / r.norm()))


def test_in_a_graph():
    b = Block(t=100, layout="kplanes").to("cuda")
    for _ in range(2):
        b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = b.step()
    for rep in range(4):
        new = Block(t=100, seed=rep + 10)
        for name in ("x", "stream_in", "dout"):
            getattr(b, name).copy_(getattr(new, name))
        for v in out.values():
            v.view(torch.uint8).fill_(0x5A + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager, _ = b.step()
        torch.cuda.synchronize()
        for name, v in out.items():
            assert torch.equal(v, eager[name]), (rep, name)
    del graph


def test_two_graphs_replayed_side_by_side():
    bs = [Block(t=700, seed=i).to("cuda") for i in (1, 2)]
    want = [b.step()[0] for b in bs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in bs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.step()[0])
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
    bs = [Block(t=400, seed=i).to("cuda") for i in (3, 4)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    want = [b.step(stream=torch.cuda.current_stream())[0] for b in bs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [b.step(stream=s)[0] for b, s in zip(bs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for name in g:
                assert torch.equal(g[name], w[name]), name
    raw, _ = bs[0].step(stream=streams[0].cuda_stream)
    streams[0].synchronize()
    for name in raw:
        assert torch.equal(raw[name], want[0][name])


def test_results_do_not_depend_on_the_run():
    b = Block(t=2000, e=64, k=6, groups=8, top_groups=3).to("cuda")
    first, _ = b.step()
    for _ in range(5):
        again, _ = b.step()
        for name in first:
            assert torch.equal(first[name], again[name]), name


def test_norm_rows_into_the_grouped_product():
    """The norm's MX rows are moegg_run's A and SFA: a dense product of one group equals the one of dispatch's rows."""
    import synth
    t, kk, n = 256, 512, 96
    gen = torch.Generator().manual_seed(3)
    x, w = torch.randn(t, kk, generator=gen).to(BF).cuda(), torch.rand(kk, generator=gen).cuda() + 0.5
    b, sfb = (torch.from_numpy(v).cuda() for v in synth.mx_quantize((torch.randn(1, n, kk, generator=gen) / 20).numpy(), "e4m3"))
    codes, sf = mg.rms_norm(x, w, dtype="e4m3")
    po = torch.tensor([t], dtype=torch.int32, device="cuda")
    d, amax = torch.empty(t, n, dtype=BF, device="cuda"), torch.empty(1, device="cuda")
    mg.run(dict(num_groups=1, valid_m=t, n=n, k=kk, ab_dtype="e4m3", d_dtype="bf16", act="none"),
           dict(a=codes, sfa=sf, b=b, sfb=sfb, padded_offsets=po, alpha=torch.ones(1, device="cuda"),
                prob=torch.ones(t, device="cuda"), d=d, amax=amax))
    av = ref.decode(codes.cpu(), sf.cpu(), "e4m3")
    bv = ref.decode(b[0].cpu(), sfb[0].cpu(), "e4m3")
    want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    # one rounding of the result; the matrix core's sums of 512 products in fp32, truncated at most
    assert ((d.cpu().double() - want).abs() <= ref.BF16 * want.abs() + 2 * 512 * ref.F32 * mag).all()


class Normed(torch.autograd.Function):
    """Residual and norm, then a gated product whose input and c are kept in 8 bits, as a user wraps them."""
    @staticmethod
    def forward(ctx, x, r, g, w, b):
        y, y8, h = mg.rms_norm(x, g, residual=r, copy="e4m3")
        z, c8 = mg.linear(y, w, bias=b, act="swiglu", save_c="e4m3")
        ctx.save_for_backward(h, g, w, *y8, *c8)
        return z, h

    @staticmethod
    def backward(ctx, dz, dh):
        h, g, w, yc, ys, cc, cs = ctx.saved_tensors
        dy, dw, db = mg.linear_backward(dz.contiguous(), (yc, ys), w, c=(cc, cs), act="swiglu", x_dtype="e4m3", c_dtype="e4m3")
        dx, dg = mg.rms_norm_backward(dy, h, g, dh=dh.contiguous())
        return dx, dx, dg, dw, db


def test_inside_a_function():
    """Gradients through torch's graph against those of the same calls without one."""
    m, n, k = 150, 192, 256
    gen = torch.Generator().manual_seed(3)
    x, r = torch.randn(m, k, generator=gen).to(BF).cuda(), torch.randn(m, k, generator=gen).to(BF).cuda()
    g, b = torch.rand(k, generator=gen).cuda() + 0.5, torch.randn(n, generator=gen).cuda() * 0.1
    w = (torch.randn(n, k, generator=gen) / math.sqrt(k)).to(BF).cuda()
    dz, dh = torch.randn(m, n // 2, generator=gen).to(BF).cuda(), torch.randn(m, k, generator=gen).to(BF).cuda()
    leaves = [t.clone().requires_grad_() for t in (x, r, g, w, b)]
    z, h = Normed.apply(*leaves)
    torch.autograd.backward([z, h], [dz, dh])
    y, y8, h0 = mg.rms_norm(x, g, residual=r, copy="e4m3")
    z0, c8 = mg.linear(y, w, bias=b, act="swiglu", save_c="e4m3")
    dy, dw, db = mg.linear_backward(dz, y8, w, c=c8, act="swiglu", x_dtype="e4m3", c_dtype="e4m3")
    dx, dg = mg.rms_norm_backward(dy, h0, g, dh=dh)
    assert torch.equal(z, z0) and torch.equal(h, h0)
    for leaf, want in zip(leaves, (dx, dx, dg, dw, db)):
        assert torch.equal(leaf.grad, want)


def test_results_have_no_history():
    x = torch.randn(12, 256, device="cuda").to(BF).requires_grad_()
    w = torch.ones(256, device="cuda").requires_grad_()
    y, (c, s), h = mg.rms_norm(x, w, residual=x, copy="e4m3")
    v = torch.randn(64, 256, device="cuda").to(BF).requires_grad_()
    z, (zc, zs) = mg.linear(x, v, save_c="e4m3")
    grads = [*mg.rms_norm_backward(x, x, w), *mg.linear_backward(z, x, v), *mg.linear_backward(z, (c, s), v, x_dtype="e4m3")]
    for t in (y, c, s, h, z, zc, zs, *mg.quantise(x), mg.dequantise((c, s)), *grads):
        assert not t.requires_grad and t.grad_fn is None
    assert x.grad is None and w.grad is None


def test_tensors_are_checked():
    x, w = torch.zeros(4, 256, dtype=BF, device="cuda"), torch.ones(256, device="cuda")

    v = torch.zeros(64, 256, dtype=BF, device="cuda")
    dy = torch.zeros(4, 64, dtype=BF, device="cuda")
    pair = mg.quantise(x)
    planes = mg.quantise(x, sf_layout="kplanes")
    for call, err in [
        (lambda: mg.rms_norm(x, w[:128]), ValueError), (lambda: mg.rms_norm(x, w.to(BF)), TypeError),
        (lambda: mg.rms_norm(x, w.cpu()), ValueError), (lambda: mg.rms_norm(x.t(), w), ValueError),
        (lambda: mg.rms_norm(x[0], w), ValueError), (lambda: mg.rms_norm(x, w, residual=x[:3]), ValueError),
        (lambda: mg.rms_norm(x, w, residual=x.half()), TypeError), (lambda: mg.rms_norm(x, w, residual=[1]), TypeError),
        (lambda: mg.rms_norm(x.float(), w, residual=x), mg.MoeggError), (lambda: mg.rms_norm(x, w, eps=0.0), mg.MoeggError),
        (lambda: mg.rms_norm(x, w, residual=x, h=torch.empty(4, 256, device="cuda")), TypeError),
        (lambda: mg.rms_norm(x, w, residual=torch.zeros_like(x), h=x), mg.MoeggError),
        (lambda: mg.rms_norm(x[:, :128].contiguous(), w[:128].contiguous(), dtype="e2m1x2"), mg.MoeggError),
        (lambda: mg.rms_norm(torch.zeros(2, 12, dtype=BF, device="cuda"), torch.ones(12, device="cuda")), mg.MoeggError),
        (lambda: mg.rms_norm_backward(x.float(), x, w), TypeError), (lambda: mg.rms_norm_backward(x, x, w, dh=x.float()), TypeError),
        (lambda: mg.rms_norm_backward(x[:2], x, w), ValueError),
        (lambda: mg.route(x, 2, num_groups=3, top_groups=2), mg.MoeggError),
        (lambda: mg.route(x, 40, num_groups=8, top_groups=1), mg.MoeggError),
        (lambda: mg.quantise(x[:, ::2]), ValueError), (lambda: mg.quantise(x, out=pair[0]), TypeError),
        (lambda: mg.quantise(x, out=(pair[0], planes[1])), ValueError),
        (lambda: mg.dequantise(planes), ValueError), (lambda: mg.dequantise(pair, sf_layout="kplanes"), ValueError),
        (lambda: mg.dequantise((pair[0], pair[1].cpu())), ValueError),
        (lambda: mg.linear(x, v[:40].contiguous(), save_c="e4m3"), mg.MoeggError),
        (lambda: mg.linear_backward(dy, pair, v), TypeError), (lambda: mg.linear_backward(dy, x, v, x_dtype="e4m3"), TypeError),
        (lambda: mg.linear_backward(dy, planes, v, x_dtype="e4m3"), ValueError),
        (lambda: mg.linear_backward(dy, (pair[0], pair[1].float()), v, x_dtype="e4m3"), TypeError),
        (lambda: mg.linear_backward(dy, pair, v, act="gelu", x_dtype="e4m3", c_dtype="e4m3"), ValueError),
        (lambda: mg.linear_backward(dy, pair, v, c=pair, act="gelu", x_dtype="e4m3", c_dtype="e4m3"), ValueError),
    ]:
        with pytest.raises(err):
            call()
