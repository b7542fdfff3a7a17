"""More operators of an MoE layer, as they are measured.

Three operators, each in its plain form (elementary torch operations in 32
bits, 64 where a choice hangs on the last bit) and, where ``own`` is true,
through the library's entry points:

* ``norm``    root-mean-square norm with the residual's addition, its output in
              BF16, in 8 bits with scales or both, and its gradient
* ``route``   the router that chooses groups of experts first, then experts of
              those groups, and its gradient
* ``saved``   activations kept in 8 bits: rows brought to MX form and back, the
              matrix product that keeps its pre-activation so, and its gradients
              from an input and a pre-activation in 8 bits

``exact`` gives the outputs again in 64 bits, from the definitions.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715
EPS = 1e-6
Q_MAX = {"e4m3": 448.0, "e5m2": 57344.0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a handful of sequences: the layer's entry, where latency counts
        _norm("norm_decode", way="forward", rows=5, width=2048, stream="bfloat16", residual=True, out="bf16", copy=None,
              layout="row_major"),
        # prompt processing in 8 bits: the norm writes the grouped product's operand itself; an odd number of tokens
        _norm("norm_mxfp8", way="forward", rows=4999, width=4096, stream="bfloat16", residual=True, out="e4m3",
              copy=None, layout="kplanes"),
        # a training batch with the residual stream in 32 bits: BF16 for the products, 8 bits kept for their gradients
        _norm("norm_train", way="forward", rows=16381, width=2048, stream="float32", residual=True, out="bf16",
              copy="e4m3", layout="row_major"),
        # its gradient, with the one that comes along the stream
        _norm("norm_grad", way="backward", rows=16381, width=2048, stream="bfloat16", residual=True, out="bf16",
              copy=None, layout="row_major"),
        # a handful of tokens, 3 of 8 groups by their best expert
        _route("groups_decode", tokens=5, experts=64, top_k=6, groups=8, top_groups=3, best=1, score="softmax",
               renormalise=True, bias=False, dtype="float32", grad=False),
        # a training batch over many experts: 4 of 8 groups by their two best, a balancing bias that steers the choice
        # only, some experts masked, some tokens (padding) with every expert masked; an odd number of tokens
        _route("groups_train", tokens=16381, experts=256, top_k=8, groups=8, top_groups=4, best=2, score="sigmoid",
               renormalise=True, bias=True, dtype="bfloat16", grad=True),
        # rows to 8 bits and back: what a checkpoint costs where no operator writes it itself
        _saved("saved_rows", way="rows", rows=16384, n=0, k=2048, experts=0, act="none", fmt="e4m3", layout="row_major"),
        # a gated first product of a few sequences that keeps its pre-activation in 8 bits
        _saved("saved_forward_small", way="forward", rows=193, n=2816, k=2048, experts=0, act="swiglu", fmt="e4m3",
               layout="row_major"),
        # the same at a training batch
        _saved("saved_forward", way="forward", rows=16384, n=2816, k=2048, experts=0, act="swiglu", fmt="e4m3",
               layout="row_major"),
        # gradients of a few rows: latency of the chain of launches
        _saved("saved_grad_small", way="backward", rows=129, n=512, k=512, experts=0, act="gelu", fmt="e5m2",
               layout="row_major"),
        # the gated first product's gradients at the training batch, input and pre-activation in 8 bits
        _saved("saved_grad", way="backward", rows=16384, n=2816, k=2048, experts=0, act="swiglu", fmt="e4m3",
               layout="row_major"),
        # the experts' gradients from the grouped product's own 8-bit operand; ragged groups, some empty
        _saved("saved_experts_grad", way="backward", rows=24571, n=1408, k=2048, experts=64, act="swiglu", fmt="e4m3",
               layout="kplanes"),
    ]


def _norm(name, **kw):
    return {"name": name, "op": "norm", **kw}


def _route(name, **kw):
    return {"name": name, "op": "route", **kw}


def _saved(name, **kw):
    return {"name": name, "op": "saved", **kw}


def _spread(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "route", "saved", "saved", "saved"))
    if op == "norm":
        out = rng.choice(("bf16", "bf16", "e4m3", "e5m2"))
        way = rng.choice(("forward", "forward", "backward"))
        width = 128 * _spread(rng, 1, 64) if out != "bf16" or rng.random() < 0.4 else 8 * _spread(rng, 2, 1024)
        return {"op": op, "way": way, "rows": _spread(rng, 1, min(16384, (16384 * 2048) // width)), "width": width,
                "stream": rng.choice(("bfloat16", "float32")), "residual": rng.random() < 0.7, "out": out,
                "copy": rng.choice((None, "e4m3", "e5m2")) if out == "bf16" and width % 128 == 0 else None,
                "layout": rng.choice(("row_major", "kplanes"))}
    if op == "route":
        groups = rng.choice((2, 4, 5, 8, 16))
        size = _spread(rng, 2, 512 // groups)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(12, top_groups * size))
        return {"op": op, "tokens": min(_spread(rng, 1, 16384), (16381 * 256) // (groups * size)),
                "experts": groups * size, "top_k": top_k, "groups": groups, "top_groups": top_groups,
                "best": rng.choice((1, 2)), "score": rng.choice(("softmax", "sigmoid")),
                # a single weight that is normalised is 1, and its gradient nothing but rounding
                "renormalise": top_k > 1 and rng.random() < 0.6, "bias": rng.random() < 0.6,
                "dtype": rng.choice(("float32", "bfloat16")), "grad": rng.random() < 0.5}
    way = rng.choice(("rows", "forward", "forward", "backward", "backward"))
    fmt, layout = rng.choice(("e4m3", "e4m3", "e5m2")), rng.choice(("row_major", "kplanes"))
    if way == "rows":
        k = 128 * _spread(rng, 1, 64) if layout == "kplanes" else 32 * _spread(rng, 1, 256)
        return {"op": op, "way": way, "rows": _spread(rng, 1, min(16384, (16384 * 2048) // k)), "n": 0, "k": k,
                "experts": 0, "act": "none", "fmt": fmt, "layout": layout}
    experts = rng.choice((0, 0, _spread(rng, 2, 64)))
    act = rng.choice(("swiglu", "swiglu", "srelu", "gelu"))
    n = 64 * rng.randint(1, 44) if act == "swiglu" else 32 * rng.randint(1, 88)
    k = 128 * rng.randint(1, 22) if way == "backward" and layout == "kplanes" else 32 * _spread(rng, 4, 88)
    most = (16384 * 2816 * 2048) // (n * k)
    return {"op": op, "way": way, "rows": _spread(rng, 1, max(1, min(16384, most))), "n": n, "k": k,
            "experts": experts, "act": act, "fmt": fmt, "layout": layout}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _bf16(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device=DEV).mul_(scale).to(torch.bfloat16)


def _channels(gen, rows, width):
    """Activations with a few large channels, as in earnest (32 bits)."""
    x = torch.randn(rows, width, generator=gen, device=DEV)
    return x.mul_(torch.exp(torch.randn(1, width, generator=gen, device=DEV)))


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "norm":
        t, h = c["rows"], c["width"]
        kind = getattr(torch, c["stream"])
        s["weight"] = torch.rand(h, generator=gen, device=DEV) + 0.5
        if c["way"] == "forward":
            # a branch's output is BF16; without a residual the stream itself comes in
            s["x"] = _channels(gen, t, h).to(torch.bfloat16 if c["residual"] else kind)
            s["residual"] = _channels(gen, t, h).mul_(4.0).to(kind) if c["residual"] else None
        else:
            s["h"] = _channels(gen, t, h).mul_(4.0).to(kind)
            s["dy"] = _bf16(gen, t, h)
            s["dh"] = torch.randn(t, h, generator=gen, device=DEV).to(kind) if c["residual"] else None
    elif c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        x = torch.randn(t, e, generator=gen, device=DEV) * 1.5
        if c["grad"]:
            if e >= 4 * k:                                                # experts out of service for some tokens
                x[torch.rand(t, e, generator=gen, device=DEV) < 0.05] = -math.inf
            x[torch.rand(t, generator=gen, device=DEV) < 0.02] = -math.inf    # padding tokens
        s["logits"] = x.to(getattr(torch, c["dtype"]))
        s["bias"] = torch.randn(e, generator=gen, device=DEV) * 0.1 if c["bias"] else None
        s["dweights"] = torch.randn(t, k, generator=gen, device=DEV)
    else:
        m, n, k, groups = c["rows"], c["n"], c["k"], max(1, c["experts"])
        if c["way"] == "rows":
            s["x"] = _channels(gen, m, k).to(torch.bfloat16)
            return s
        s["w"] = _bf16(gen, *((groups, n, k) if c["experts"] else (n, k)), scale=1.0 / math.sqrt(k))
        s["offsets"], s["most"] = None, m
        if c["experts"]:                                                  # ragged groups, some of them empty
            share = torch.rand(groups, generator=gen, device=DEV).double() ** 2
            share[torch.rand(groups, generator=gen, device=DEV) < 0.1] = 0.0
            share[-1] += 1e-3
            ends = torch.round(torch.cumsum(share, 0) / share.sum() * m).to(torch.int32)
            ends[-1] = m
            s["offsets"] = ends
            s["most"] = int(torch.diff(ends, prepend=ends.new_zeros(1)).max())
        if c["way"] == "forward":
            s["x"] = _bf16(gen, m, k)
            s["bias"] = torch.randn(*((groups, n) if c["experts"] else (n,)), generator=gen, device=DEV) * 0.2
        else:
            # what the forward pass kept: codes and scale bytes of both
            codes, byte = _plain_mx(torch.randn(m, k, generator=gen, device=DEV), c["fmt"])
            s["x"] = codes.view(torch.uint8), _planes(byte) if c["layout"] == "kplanes" else byte
            codes, byte = _plain_mx(torch.randn(m, n, generator=gen, device=DEV), c["fmt"])
            s["c"] = codes.view(torch.uint8), byte
            s["dy"] = _bf16(gen, m, n // 2 if c["act"] == "swiglu" else n)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_mx(rows, fmt):
    """Values in 8 bits and E8M0 scale bytes of blocks of 32: the smallest power of two that keeps a block in range."""
    v = rows.float().reshape(rows.shape[0], -1, 32)
    mant, expo = torch.frexp(v.abs().amax(2).double() / Q_MAX[fmt])       # mant in [0.5, 1)
    expo = torch.where(mant == 0.5, expo - 1, expo).clamp(-127, 127)
    expo = torch.where(mant == 0.0, -127, expo)
    v = (v.double() / torch.exp2(expo.double())[:, :, None]).float().reshape(rows.shape)
    return v.to(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2), (expo + 127).to(torch.uint8)


def _planes(byte):
    """(rows, blocks) scale bytes as K-block planes (blocks / 4, rows, 4)."""
    return byte.reshape(byte.shape[0], -1, 4).transpose(0, 1).contiguous()


def _factors(byte, layout):
    """Scale bytes of either layout as factors (rows, blocks)."""
    if layout == "kplanes":
        byte = byte.transpose(0, 1).reshape(byte.shape[1], -1)
    return torch.exp2(byte.double() - 127.0).float()


def _plain_values(pair, fmt, layout):
    """What codes and scale bytes stand for, in 32 bits."""
    codes, byte = pair
    v = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).float()
    return (v.reshape(v.shape[0], -1, 32) * _factors(byte, layout)[:, :, None]).reshape(v.shape)


def _mx_out(rows, fmt, layout):
    values, byte = _plain_mx(rows, fmt)
    return values, (_planes(byte) if layout == "kplanes" else byte).view(torch.float8_e8m0fnu)


def _plain_norm(s, c):
    w = s["weight"]
    if c["way"] == "backward":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        x, g = h * r, dy * w
        dx = r * (g - x * (g * x).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dw": (dy * x).sum(0)}
    out, h = {}, s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(s["residual"].dtype)   # the norm goes on with what is kept
        out["h"] = h
    h = h.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w
    if c["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    mx = c["copy"] if c["out"] == "bf16" else c["out"]
    if mx:
        out["codes"], out["scales"] = _mx_out(y, mx, c["layout"])
    return out


def _plain_route(s, c):
    t, e, k, groups = c["tokens"], c["experts"], c["top_k"], c["groups"]
    x = s["logits"].float().clamp(max=torch.finfo(torch.float32).max)
    top = x.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    if c["score"] == "softmax":
        p = torch.exp(x - top)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = x
    if c["bias"] or c["best"] > 1:
        # the choice hangs on the last bits of sums: in 64 bits
        if c["score"] == "softmax":
            exact = torch.exp((x - top).double())
            exact = exact / exact.sum(1, keepdim=True).clamp(min=1e-300)
        else:
            exact = 1.0 / (1.0 + torch.exp(-x.double()))
        score = exact + s["bias"].double() if c["bias"] else exact
        score = torch.where(x == -math.inf, -math.inf, score)
        key = score if c["bias"] else x
    else:
        score = x
    best = torch.sort(score.reshape(t, groups, -1), dim=2, descending=True)[0][:, :, :c["best"]]
    some = best[:, :, 0] != -math.inf
    total = torch.where(best == -math.inf, 0.0, best).sum(2)
    order = torch.sort(torch.where(some, total, -math.inf), dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
    in_group = torch.zeros(t, groups, dtype=torch.bool, device=x.device).scatter_(1, order, True)
    key = torch.where(in_group.repeat_interleave(e // groups, 1), key, -math.inf)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)       # ties: lowest index first
    key, ids = key[:, :k], ids[:, :k]
    there = key != -math.inf
    w = torch.where(there, p.gather(1, ids), 0.0)
    total = w.sum(1, keepdim=True).clamp(min=1e-30)
    if c["renormalise"]:
        w = w / total
    ids32 = torch.where(there, ids, -1).to(torch.int32)
    if not c["grad"]:
        return {"ids": ids32, "weights": w}
    g = torch.where(there, s["dweights"], 0.0)
    if c["renormalise"]:
        gs = (g - (g * w).sum(1, keepdim=True)) / total                   # gradient of the chosen scores
        gs = torch.where(there, gs, 0.0)
    else:
        gs = g
    full = torch.zeros_like(p).scatter_add_(1, ids, gs)
    if c["score"] == "softmax":
        d = p * (full - (full * p).sum(1, keepdim=True))
    else:
        d = full * p * (1.0 / (1.0 + torch.exp(x)))
    return {"ids": ids32, "weights": w, "dlogits": d.to(s["logits"].dtype)}


def _plain_act(z, act):
    if act == "swiglu":
        v = z.reshape(z.shape[0], -1, 2, 32)
        return (v[:, :, 0] * (v[:, :, 1] / (1.0 + torch.exp(-v[:, :, 1])))).reshape(z.shape[0], -1)
    if act == "srelu":
        return torch.clamp(z, min=0.0) ** 2
    return 0.5 * z * (1.0 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))


def _plain_dact(dy, z, act):
    if act == "swiglu":
        v, d = z.reshape(z.shape[0], -1, 2, 32), dy.reshape(z.shape[0], -1, 32)
        sig = 1.0 / (1.0 + torch.exp(-v[:, :, 1]))
        return torch.stack([d * v[:, :, 1] * sig, d * v[:, :, 0] * sig * (1.0 + v[:, :, 1] * (1.0 - sig))],
                           2).reshape(z.shape)
    if act == "srelu":
        return dy * 2.0 * torch.clamp(z, min=0.0)
    t = torch.tanh(GELU_C * (z + GELU_A * z * z * z))
    return dy * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * z * z))


def _plain_saved(s, c):
    if c["way"] == "rows":
        codes, scales = _mx_out(s["x"], c["fmt"], c["layout"])
        pair = codes.view(torch.uint8), scales.view(torch.uint8)
        return {"codes": codes, "scales": scales, "x": _plain_values(pair, c["fmt"], c["layout"]).to(torch.bfloat16)}
    w, m = s["w"].float(), c["rows"]
    if s["offsets"] is not None:                                          # every group's rows, padded to the longest's
        ends = s["offsets"].long()
        row = torch.cat([ends.new_zeros(1), ends[:-1]])[:, None] + torch.arange(s["most"], device=ends.device)
        mine = (row < ends[:, None])[:, :, None]
        row = row.clamp(max=m - 1)
        group = (torch.arange(m, device=row.device)[:, None] >= ends).sum(1)
        at = torch.arange(m, device=row.device) - row[group, 0]
    if c["way"] == "forward":
        x = s["x"].float()
        if s["offsets"] is None:
            z = x @ w.t() + s["bias"]
        else:
            z = torch.bmm(x[row], w.transpose(1, 2).contiguous())[group, at] + s["bias"][group]
        codes, scales = _mx_out(z, c["fmt"], "row_major")
        return {"y": _plain_act(z, c["act"]).to(torch.bfloat16), "c": codes, "scales": scales}
    x = _plain_values(s["x"], c["fmt"], c["layout"])
    dz = _plain_dact(s["dy"].float(), _plain_values(s["c"], c["fmt"], "row_major"), c["act"])
    if s["offsets"] is None:
        return {"dx": (dz @ w).to(torch.bfloat16), "dw": (dz.t() @ x).to(torch.bfloat16), "db": dz.sum(0)}
    dzg, xg = torch.where(mine, dz[row], 0.0), torch.where(mine, x[row], 0.0)
    return {"dx": torch.bmm(dzg, w)[group, at].to(torch.bfloat16),
            "dw": torch.bmm(dzg.transpose(1, 2).contiguous(), xg).to(torch.bfloat16), "db": dzg.sum(1)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(codes, scales, fmt):
    """The library's codes and scale bytes under the types of what they stand for."""
    return (codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2),
            scales.view(torch.float8_e8m0fnu))


def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "route": _plain_route, "saved": _plain_saved}[c["op"]](s, c)
    import moe_grouped_block_amd as mg
    if c["op"] == "norm":
        if c["way"] == "backward":
            dx, dw = mg.rms_norm_backward(s["dy"], s["h"], s["weight"], dh=s["dh"], eps=EPS)
            return {"dx": dx, "dw": dw}
        got = mg.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, dtype=c["out"], copy=c["copy"],
                          sf_layout=c["layout"])
        got, out = list(got) if s["residual"] is not None or c["copy"] else [got], {}
        if s["residual"] is not None:
            out["h"] = got.pop()
        if c["out"] == "bf16":
            out["y"] = got.pop(0)
        if got:
            out["codes"], out["scales"] = _values(*got[0], c["copy"] if c["out"] == "bf16" else c["out"])
        return out
    if c["op"] == "route":
        how = dict(score=c["score"], renormalise=c["renormalise"])
        ids, weights = mg.route(s["logits"], c["top_k"], bias=s["bias"], num_groups=c["groups"],
                                top_groups=c["top_groups"], group_best=c["best"], **how)
        out = {"ids": ids, "weights": weights}
        if c["grad"]:
            out["dlogits"] = mg.route_backward(s["logits"], ids, s["dweights"], **how)
        return out
    if c["way"] == "rows":
        pair = mg.quantise(s["x"], dtype=c["fmt"], sf_layout=c["layout"])
        back = mg.dequantise(pair, dtype=c["fmt"], sf_layout=c["layout"])
        codes, scales = _values(*pair, c["fmt"])
        return {"codes": codes, "scales": scales, "x": back}
    if c["way"] == "forward":
        y, pair = mg.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], offsets=s["offsets"], save_c=c["fmt"])
        codes, scales = _values(*pair, c["fmt"])
        return {"y": y, "c": codes, "scales": scales}
    dx, dw, db = mg.linear_backward(s["dy"], s["x"], s["w"], c=s["c"], act=c["act"], offsets=s["offsets"],
                                    x_dtype=c["fmt"], c_dtype=c["fmt"], sf_layout=c["layout"])
    return {"dx": dx, "dw": dw, "db": db}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(c):
    if c["op"] == "norm":
        n, size = c["rows"] * c["width"], 4 if c["stream"] == "float32" else 2
        if c["way"] == "backward":
            return {"bytes": n * (2 + size * (3 if c["residual"] else 2)) + c["width"] * 8, "flops": 14 * n}
        moved = 2 + 2 * size if c["residual"] else size
        mx = c["copy"] if c["out"] == "bf16" else c["out"]
        moved += (2 if c["out"] == "bf16" else 0) + (33 / 32 if mx else 0)
        return {"bytes": int(n * moved) + c["width"] * 4, "flops": 6 * n}
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        size = 4 if c["dtype"] == "float32" else 2
        # the gradient is a call of its own: it reads the chosen logits and writes a row for every token
        return {"bytes": t * e * size * (2 if c["grad"] else 1) + t * k * (20 if c["grad"] else 8),
                "flops": t * e * (10 if c["grad"] else 6)}
    m, n, k, groups = c["rows"], c["n"], c["k"], max(1, c["experts"])
    if c["way"] == "rows":
        return {"bytes": m * k * 2 + 2 * (m * k * 33 // 32) + m * k * 2, "flops": 6 * m * k}
    n_out, weights = n // 2 if c["act"] == "swiglu" else n, min(groups, m) * n * k
    if c["way"] == "forward":
        return {"bytes": 2 * (m * k + weights + m * n_out) + m * n * 33 // 32 + 4 * groups * n, "flops": 2 * m * n * k}
    return {"bytes": 2 * (weights + m * n_out + m * k + groups * n * k) + m * (n + k) * 33 // 32 + 4 * groups * n,
            "flops": 4 * m * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"norm": _exact_norm, "route": _exact_route, "saved": _exact_saved}[c["op"]](s, c)


def _exact_mx(v, fmt, layout):
    """Values on their grids and scales of rows in 64 bits."""
    bits, low, most = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    rows, width = v.shape
    v = v.reshape(rows, width // 32, 32)
    amax = v.abs().amax(2)
    scale = torch.full_like(amax, 2.0 ** -127)
    for power in range(-126, 128):                                        # the smallest power of two that is enough
        scale = torch.where(amax > scale * most, 2.0 ** power, scale)
    v = v / scale[:, :, None]
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    v = (torch.round(v / unit) * unit).reshape(rows, width)               # torch.round: ties to even
    if layout == "kplanes":
        scale = scale.reshape(rows, width // 128, 4).permute(1, 0, 2).contiguous()
    return v, scale


def _exact_norm(s, c):
    w = s["weight"].double()
    if c["way"] == "backward":
        # through the norm's own Jacobian: y_i = w_i h_i (q / n + eps)^(-1/2), q = sum h^2
        h, dy, n = s["h"].double(), s["dy"].double(), c["width"]
        q = (h ** 2).sum(1, keepdim=True) / n + EPS
        dx = dy * w / torch.sqrt(q) - h * (dy * w * h).sum(1, keepdim=True) / (n * q ** 1.5)
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": (dy * h / torch.sqrt(q)).sum(0)}
    out, h = {}, s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
        out["h"] = h
        h = h.to(s["residual"].dtype).double()
    y = h / torch.sqrt((h ** 2).sum(1, keepdim=True) / c["width"] + EPS) * w
    if c["out"] == "bf16":
        out["y"] = y
    mx = c["copy"] if c["out"] == "bf16" else c["out"]
    if mx:
        out["codes"], out["scales"] = _exact_mx(y, mx, c["layout"])
    return out


def _exact_route(s, c):
    x = s["logits"].cpu().double().numpy()
    t, e = x.shape
    size = e // c["groups"]
    with np.errstate(all="ignore"):
        finite = np.where(np.isneginf(x).all(1, keepdims=True), 0.0, x)
        if c["score"] == "softmax":
            ex = np.exp(finite - finite.max(1, keepdims=True))
            p = np.where(np.isneginf(x), 0.0, ex / ex.sum(1, keepdims=True))
        else:
            p = np.exp(-np.logaddexp(0.0, -x))
        score = p + s["bias"].cpu().double().numpy() if c["bias"] else (p if c["best"] > 1 else x.copy())
        score = np.where(np.isneginf(x), -np.inf, score)
        left = np.where(np.isneginf(x), -np.inf, score if c["bias"] else x)
    every = np.arange(t)
    parts = score.reshape(t, c["groups"], size)
    total = np.full((t, c["groups"]), -np.inf)
    rest = parts.copy()
    for _ in range(min(c["best"], size)):                                 # the best that is left, added
        top = rest.max(2)
        total = np.where(top > -np.inf, np.where(total > -np.inf, total, 0.0) + np.where(top > -np.inf, top, 0.0), total)
        at = rest.argmax(2)
        np.put_along_axis(rest, at[:, :, None], -np.inf, 2)
    closed = np.ones((t, c["groups"]), bool)
    for _ in range(c["top_groups"]):
        g = total.argmax(1)
        closed[every[total[every, g] > -np.inf], g[total[every, g] > -np.inf]] = False
        total[every, g] = -np.inf
    left = np.where(np.repeat(closed, size, 1), -np.inf, left)
    ids = np.full((t, c["top_k"]), -1, np.int64)
    w = np.zeros((t, c["top_k"]))
    for j in range(c["top_k"]):                                           # the largest that is left, lowest index first
        best = left.argmax(1)
        there = left[every, best] > -np.inf
        ids[there, j], w[there, j] = best[there], p[every, best][there]
        left[every, best] = -np.inf
    chosen = w.copy()
    if c["renormalise"]:
        sums = chosen.sum(1, keepdims=True)
        w = np.divide(chosen, sums, out=np.zeros_like(chosen), where=sums > 0)
    out = {"ids": ids.astype(np.int32), "weights": w}
    if c["grad"]:
        # through the weights' own Jacobian: d w_i / d s_j, then d s_j / d logit
        g = np.where(ids >= 0, s["dweights"].cpu().double().numpy(), 0.0)
        ds = g
        if c["renormalise"]:
            ds = np.divide(g * sums - (g * chosen).sum(1, keepdims=True), sums * sums, out=np.zeros_like(g),
                           where=sums > 0) * (ids >= 0)
        full = np.zeros((t, e))
        np.add.at(full, (every[:, None], np.maximum(ids, 0)), ds)
        if c["score"] == "softmax":
            out["dlogits"] = p * full - p * (p * full).sum(1, keepdims=True)
        else:
            out["dlogits"] = full * p * (1.0 - p)
    return out


def _exact_saved(s, c):
    def value(pair, layout):
        """Codes taken apart by their bits."""
        code, byte = pair[0].long(), pair[1].double()
        bits, bias = (3, 7) if c["fmt"] == "e4m3" else (2, 15)
        expo, mant = (code & 127) >> bits, (code & (2 ** bits - 1)).double() / 2 ** bits
        v = torch.where(expo > 0, (1.0 + mant) * torch.exp2((expo - bias).double()), mant * 2.0 ** (1 - bias))
        v = torch.where(code > 127, -v, v)
        if layout == "kplanes":
            byte = byte.permute(1, 0, 2).reshape(v.shape[0], -1)
        return v * torch.exp2(byte - 127.0).repeat_interleave(32, 1)

    if c["way"] == "rows":
        v, scale = _exact_mx(s["x"].double(), c["fmt"], "row_major")
        out = {"codes": v, "scales": scale, "x": v * scale.repeat_interleave(32, 1)}
        if c["layout"] == "kplanes":
            out["scales"] = scale.reshape(scale.shape[0], -1, 4).permute(1, 0, 2).contiguous()
        return out
    m, n, act = c["rows"], c["n"], c["act"]
    ends = [m] if s["offsets"] is None else s["offsets"].cpu().tolist()
    w = s["w"] if s["w"].dim() == 3 else s["w"][None]
    linear = torch.arange(n, device=DEV).reshape(-1, 64)[:, :32].reshape(-1) if act == "swiglu" else None
    if c["way"] == "forward":
        bias, parts, at = s["bias"].reshape(len(ends), n).double(), [], 0
        for g, end in enumerate(ends):
            parts.append(s["x"][at:end].double() @ w[g].double().t() + bias[g])
            at = end
        z = torch.cat(parts, 0)
        if act == "swiglu":
            y = z[:, linear] * z[:, linear + 32] * torch.sigmoid(z[:, linear + 32])
        elif act == "srelu":
            y = torch.where(z > 0, z * z, 0.0)
        else:
            y = z * torch.sigmoid(2.0 * GELU_C * (z + GELU_A * z ** 3))
        v, scale = _exact_mx(z, c["fmt"], "row_major")
        return {"y": y, "c": v, "scales": scale}
    x, z, d = value(s["x"], c["layout"]), value(s["c"], "row_major"), s["dy"].double()
    if act == "swiglu":
        lin, gate = z[:, linear], z[:, linear + 32]
        sig, dz = torch.sigmoid(gate), torch.empty_like(z)
        dz[:, linear] = d * gate * sig
        dz[:, linear + 32] = d * lin * (sig + gate * sig * torch.sigmoid(-gate))
    elif act == "srelu":
        dz = torch.where(z > 0, 2.0 * z * d, 0.0)
    else:
        sig = torch.sigmoid(2.0 * GELU_C * (z + GELU_A * z ** 3))
        dz = d * (sig + z * sig * (1.0 - sig) * 2.0 * GELU_C * (1.0 + 3.0 * GELU_A * z ** 2))
    dx, dw, db, at = [], [], [], 0
    for g, end in enumerate(ends):
        dx.append(dz[at:end] @ w[g].double())
        dw.append(dz[at:end].t() @ x[at:end])
        db.append(dz[at:end].sum(0))
        at = end
    return {"dx": torch.cat(dx, 0), "dw": torch.stack(dw).reshape(s["w"].shape),
            "db": torch.stack(db) if s["offsets"] is not None else db[0]}
