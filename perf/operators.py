"""The operators around the experts' products, as they are measured.

Three operators of an MoE layer, each in its plain form (elementary torch
operations in 32 bits, 64 where a choice hangs on the last bit) and, where
``own`` is true, through the library's entry points:

* ``route``     router scores, the top-k choice and its gradient
* ``exchange``  tokens sorted by expert and back, with the weights applied,
                and the gradients of both ways
* ``linear``    the matrix product with bias, activation and residual in its
                epilogue, dense or grouped by expert, and its gradients

``exact`` gives every output again in 64 bits, from the definitions.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a handful of sequences: latency is what counts
        _route("route_decode", tokens=5, experts=64, top_k=6, score="softmax", renormalise=True, bias=False,
               dtype="float32", grad=False),
        # a training batch over many experts with a balancing bias that steers the choice only; some
        # experts masked, some tokens (padding) with every expert masked; an odd number of tokens
        _route("route_train", tokens=16381, experts=256, top_k=8, score="sigmoid", renormalise=True, bias=True,
               dtype="bfloat16", grad=True),
        # the same decoding step: sort, gather, combine for three tokens, experts' rows unpadded
        _exchange("exchange_decode", way="forward", tokens=3, experts=64, top_k=6, width=2048, m_aligned=1,
                  fmt="bf16", drop=False),
        # prompt processing at 16384 tokens, top-6 of 64: rows padded to the grouped product's 128
        _exchange("exchange_prompt", way="forward", tokens=16384, experts=64, top_k=6, width=2048, m_aligned=128,
                  fmt="bf16", drop=False),
        # the gather that also writes MXFP8 operands for the grouped product; odd token count, padding tokens
        _exchange("exchange_mxfp8", way="quantise", tokens=4999, experts=32, top_k=4, width=4096, m_aligned=128,
                  fmt="e4m3", drop=True),
        # the gradients of both ways at the training batch
        _exchange("exchange_grad", way="backward", tokens=16384, experts=64, top_k=6, width=2048, m_aligned=128,
                  fmt="bf16", drop=False),
        # one token through a gated first product: the weights are read once, nothing else matters
        _linear("linear_decode", way="forward", rows=1, n=2816, k=2048, experts=0, act="swiglu", bias=True,
                residual=False, save_c=False, out="bfloat16"),
        # 96 routed rows over 64 experts (16 tokens, top-6): a few rows for each expert, second product
        _linear("linear_experts_decode", way="forward", rows=96, n=2048, k=1408, experts=64, act="none", bias=True,
                residual=False, save_c=False, out="bfloat16"),
        # the router's product: a narrow output in 32 bits
        _linear("linear_router", way="forward", rows=16384, n=64, k=2048, experts=0, act="none", bias=True,
                residual=False, save_c=False, out="float32"),
        # a dense (shared) block's second product with the routed sum as its residual; an odd number of rows
        _linear("linear_residual", way="forward", rows=4099, n=2048, k=2816, experts=0, act="gelu", bias=True,
                residual=True, save_c=True, out="bfloat16"),
        # the gated first product's gradients at the training batch
        _linear("linear_grad", way="backward", rows=16384, n=2816, k=2048, experts=0, act="swiglu", bias=True,
                residual=False, save_c=False, out="bfloat16"),
        # the experts' gradients with 32-bit weight gradients; ragged groups, some empty
        _linear("linear_experts_grad", way="backward", rows=24571, n=2048, k=1408, experts=64, act="none", bias=True,
                residual=False, save_c=False, out="float32"),
    ]


def _route(name, **kw):
    return {"name": name, "op": "route", **kw}


def _exchange(name, **kw):
    return {"name": name, "op": "exchange", **kw}


def _linear(name, **kw):
    return {"name": name, "op": "linear", **kw}


def _spread(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "exchange", "exchange", "linear", "linear", "linear"))
    if op == "route":
        experts = _spread(rng, 4, 512)
        top_k = rng.randint(1, min(12, experts))
        return {"op": op, "tokens": min(_spread(rng, 1, 16384), (16381 * 256) // experts), "experts": experts,
                "top_k": top_k, "score": rng.choice(("softmax", "sigmoid")),
                # a single weight that is normalised is 1, and its gradient nothing but rounding
                "renormalise": top_k > 1 and rng.random() < 0.6, "bias": rng.random() < 0.5,
                "dtype": rng.choice(("float32", "bfloat16")), "grad": rng.random() < 0.6}
    if op == "exchange":
        way = rng.choice(("forward", "quantise", "backward"))
        width = 256 * rng.randint(1, 16)
        experts, top_k = _spread(rng, 2, 256), rng.randint(1, 8)
        most = (16384 * 6 * 2048) // (top_k * width)
        return {"op": op, "way": way, "tokens": _spread(rng, 1, max(1, min(16384, most))), "experts": experts,
                "top_k": min(top_k, experts), "width": width, "m_aligned": rng.choice((1, 32, 128)),
                "fmt": rng.choice(("e4m3", "e5m2")) if way == "quantise" else "bf16", "drop": rng.random() < 0.5}
    way = rng.choice(("forward", "forward", "backward"))
    experts = rng.choice((0, 0, _spread(rng, 2, 64)))
    act = rng.choice(("none", "swiglu", "srelu", "gelu"))
    n = 64 * rng.randint(1, 44) if act == "swiglu" else 8 * _spread(rng, 2, 352)
    k = 8 * _spread(rng, 16, 352)
    most = (16384 * 2816 * 2048) // (n * k)
    return {"op": op, "way": way, "rows": _spread(rng, 1, max(1, min(16384, most))), "n": n, "k": k,
            "experts": experts, "act": act, "bias": rng.random() < 0.7,
            "residual": way == "forward" and rng.random() < 0.5, "save_c": way == "forward" and rng.random() < 0.4,
            "out": rng.choice(("bfloat16", "float32")) if way == "forward" or act == "none" else "bfloat16"}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _capacity(c):
    """Rows that any routing of the case fits into."""
    slots = c["tokens"] * c["top_k"]
    return (slots + min(slots, c["experts"]) * (c["m_aligned"] - 1)) // c["m_aligned"] * c["m_aligned"]


def _chosen(c, gen):
    """Distinct experts for every token, some experts more popular than others; -1 where a token has none."""
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    score = torch.randn(t, e, generator=gen, device=DEV) + torch.randn(1, e, generator=gen, device=DEV) * 0.5
    ids = score.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    if c["drop"]:
        ids[torch.rand(t, generator=gen, device=DEV) < 0.1] = -1          # padding tokens
        ids[torch.rand(t, k, generator=gen, device=DEV) < 0.05] = -1      # slots over an expert's capacity
    return ids


def _bf16(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device=DEV).mul_(scale).to(torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        x = torch.randn(t, e, generator=gen, device=DEV) * 1.5
        if c["grad"]:
            if e >= 4 * k:                                                # experts out of service for some tokens
                x[torch.rand(t, e, generator=gen, device=DEV) < 0.05] = -math.inf
            x[torch.rand(t, generator=gen, device=DEV) < 0.02] = -math.inf    # padding tokens
        s["logits"] = x.to(getattr(torch, c["dtype"]))
        s["bias"] = torch.randn(e, generator=gen, device=DEV) * 0.1 if c["bias"] else None
        s["dweights"] = torch.randn(t, k, generator=gen, device=DEV)
    elif c["op"] == "exchange":
        t, k, h = c["tokens"], c["top_k"], c["width"]
        cap = _capacity(c)
        s["ids"] = _chosen(c, gen)
        s["weights"] = torch.rand(t, k, generator=gen, device=DEV) * 0.5 + 0.01
        if c["way"] == "forward":
            s["x"], s["rows"] = _bf16(gen, t, h), _bf16(gen, cap, h)
            s["residual"] = _bf16(gen, t, h)
            s["buffer"] = torch.zeros(cap, h, dtype=torch.bfloat16, device=DEV)
        elif c["way"] == "quantise":
            # activations with a few large channels, as in earnest
            s["x"] = _bf16(gen, t, h).mul_(torch.exp(torch.randn(1, h, generator=gen, device=DEV))).to(torch.bfloat16)
            s["buffer"] = torch.zeros(cap, h, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros(h // 128, cap, 4, dtype=torch.uint8, device=DEV)
        else:
            s["dy"], s["rows"], s["da"] = _bf16(gen, t, h), _bf16(gen, cap, h), _bf16(gen, cap, h)
            s["buffer"] = torch.zeros(cap, h, dtype=torch.bfloat16, device=DEV)
            s["offsets"], s["row_of"], s["slot_of"] = _plain_sort(s["ids"], c)
    else:
        m, n, k, groups = c["rows"], c["n"], c["k"], max(1, c["experts"])
        n_out = n // 2 if c["act"] == "swiglu" else n
        s["x"] = _bf16(gen, m, k)
        s["w"] = _bf16(gen, *((groups, n, k) if c["experts"] else (n, k)), scale=1.0 / math.sqrt(k))
        s["bias"] = torch.randn(*((groups, n) if c["experts"] else (n,)), generator=gen, device=DEV) * 0.2 \
            if c["bias"] else None
        s["residual"] = _bf16(gen, m, n_out) if c["residual"] else None
        s["offsets"], s["most"] = None, m
        if c["experts"]:                                                  # ragged groups, some of them empty
            share = torch.rand(groups, generator=gen, device=DEV).double() ** 2
            share[torch.rand(groups, generator=gen, device=DEV) < 0.1] = 0.0
            share[-1] += 1e-3
            ends = torch.round(torch.cumsum(share, 0) / share.sum() * m).to(torch.int32)
            ends[-1] = m
            s["offsets"] = ends
            s["most"] = int(torch.diff(ends, prepend=ends.new_zeros(1)).max())
        if c["way"] == "backward":
            s["dy"] = _bf16(gen, m, n_out)
            s["c"] = _bf16(gen, m, n) if c["act"] != "none" else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_route(s, c):
    e, k = c["experts"], c["top_k"]
    x = s["logits"].float().clamp(max=torch.finfo(torch.float32).max)
    top = x.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    if c["score"] == "softmax":
        p = torch.exp(x - top)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = x
    if c["bias"]:
        # the choice hangs on the last bits of score + bias: in 64 bits
        if c["score"] == "softmax":
            key = torch.exp((x - top).double())
            key = key / key.sum(1, keepdim=True).clamp(min=1e-300)
        else:
            key = 1.0 / (1.0 + torch.exp(-x.double()))
        key = torch.where(x == -math.inf, -math.inf, key + s["bias"].double())
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


def _plain_sort(ids, c):
    """Group ends, the row of every slot and the slot of every row, in 64-bit whole numbers."""
    e, ma, cap = c["experts"], c["m_aligned"], _capacity(c)
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < e), flat, e)
    counts = (flat[:, None] == torch.arange(e + 1, device=flat.device)).sum(0)
    padded = torch.div(counts[:e] + ma - 1, ma, rounding_mode="floor") * ma
    ends = torch.cumsum(padded, 0)
    starts = torch.cat([ends - padded, ends.new_zeros(1)])
    first = torch.cumsum(counts, 0) - counts
    group, order = torch.sort(flat, stable=True)                          # slots of a group in token order
    row = starts[group] + torch.arange(flat.numel(), device=flat.device) - first[group]
    row = torch.where(group < e, row, -1)
    row_of = torch.empty_like(flat)
    row_of[order] = row
    slot_of = torch.full((cap + 1,), -1, dtype=torch.int64, device=flat.device)
    slot_of[torch.where(row >= 0, row, cap)] = order
    return ends.to(torch.int32), row_of.reshape(ids.shape).to(torch.int32), slot_of[:cap].to(torch.int32)


def _plain_gather(x, slot_of, top_k):
    """Row r of the sorted order: its token's row of x, zeros where it has none."""
    there = slot_of >= 0
    token = torch.where(there, torch.div(slot_of, top_k, rounding_mode="floor"), 0).long()
    return torch.where(there[:, None], x[token], x.new_zeros(()))


def _plain_combine(rows, row_of, weights, residual):
    there = row_of >= 0
    picked = torch.where(there[:, :, None], rows[row_of.clamp(min=0).long()].float(), 0.0)
    if weights is not None:
        picked = picked * weights[:, :, None]
    y = picked.sum(1)
    if residual is not None:
        y = y + residual.float()
    return y.to(torch.bfloat16)


def _plain_mx(rows, fmt):
    """Codes and E8M0 scales of blocks of 32: the smallest power of two that keeps the block in range."""
    most, kind = (448.0, torch.float8_e4m3fn) if fmt == "e4m3" else (57344.0, torch.float8_e5m2)
    v = rows.float().reshape(rows.shape[0], -1, 32)
    mant, expo = torch.frexp(v.abs().amax(2).double() / most)             # mant in [0.5, 1)
    expo = torch.where(mant == 0.5, expo - 1, expo).clamp(-127, 127)
    expo = torch.where(mant == 0.0, -127, expo)
    scale = torch.exp2(expo.double())
    codes = (v.double() / scale[:, :, None]).float().reshape(rows.shape).to(kind)
    return codes, (expo + 127).to(torch.uint8)


def _planes(byte):
    """(rows, blocks) scale bytes as K-block planes (blocks / 4, rows, 4)."""
    return byte.reshape(byte.shape[0], -1, 4).transpose(0, 1).contiguous()


def _plain_exchange(s, c):
    if c["way"] == "backward":
        there = s["slot_of"] >= 0
        slot = s["slot_of"].clamp(min=0).long()
        w = torch.where(there, s["weights"].reshape(-1)[slot], 0.0)
        drows = (_plain_gather(s["dy"].float(), s["slot_of"], c["top_k"]) * w[:, None]).to(torch.bfloat16)
        picked = s["rows"][s["row_of"].clamp(min=0).long()].float()
        dw = torch.where(s["row_of"] >= 0, (picked * s["dy"].float()[:, None, :]).sum(2), 0.0)
        return {"drows": drows, "dweights": dw, "dx": _plain_combine(s["da"], s["row_of"], None, None)}
    ends, row_of, slot_of = _plain_sort(s["ids"], c)
    prob = torch.where(slot_of >= 0, s["weights"].reshape(-1)[slot_of.clamp(min=0).long()], 0.0)
    plan = {"offsets": ends, "row_of": row_of, "slot_of": slot_of, "prob": prob}
    a = _plain_gather(s["x"], slot_of, c["top_k"])
    if c["way"] == "forward":
        return {**plan, "a": a, "y": _plain_combine(s["rows"], row_of, s["weights"], s["residual"])}
    codes, byte = _plain_mx(a, c["fmt"])
    return {**plan, "a": codes, "scales": _planes(byte).view(torch.float8_e8m0fnu)}


def _plain_act(z, act):
    if act == "swiglu":
        v = z.reshape(z.shape[0], -1, 2, 32)
        return (v[:, :, 0] * (v[:, :, 1] / (1.0 + torch.exp(-v[:, :, 1])))).reshape(z.shape[0], -1)
    if act == "srelu":
        return torch.clamp(z, min=0.0) ** 2
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))
    return z


def _plain_dact(dy, z, act):
    if act == "swiglu":
        v, d = z.reshape(z.shape[0], -1, 2, 32), dy.reshape(z.shape[0], -1, 32)
        sig = 1.0 / (1.0 + torch.exp(-v[:, :, 1]))
        return torch.stack([d * v[:, :, 1] * sig, d * v[:, :, 0] * sig * (1.0 + v[:, :, 1] * (1.0 - sig))],
                           2).reshape(z.shape)
    if act == "srelu":
        return dy * 2.0 * torch.clamp(z, min=0.0)
    if act == "gelu":
        t = torch.tanh(GELU_C * (z + GELU_A * z * z * z))
        return dy * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * z * z))
    return dy


def _groups(s, m):
    """Row indices (groups, most) of every group, and which of them are rows of it."""
    ends = s["offsets"].long()
    starts = torch.cat([ends.new_zeros(1), ends[:-1]])
    row = starts[:, None] + torch.arange(s["most"], device=ends.device)
    return row.clamp(max=m - 1), row < ends[:, None]


def _plain_linear(s, c):
    x, w, m = s["x"].float(), s["w"].float(), c["rows"]
    if s["offsets"] is not None:
        row, mine = _groups(s, m)
        group = (torch.arange(m, device=row.device)[:, None] >= s["offsets"].long()).sum(1)
        at = torch.arange(m, device=row.device) - row[group, 0]
    if c["way"] == "forward":
        if s["offsets"] is None:
            z = x @ w.t()
            z = z if s["bias"] is None else z + s["bias"]
        else:
            z = torch.bmm(x[row], w.transpose(1, 2).contiguous())[group, at]
            z = z if s["bias"] is None else z + s["bias"][group]
        y = _plain_act(z, c["act"])
        y = y if s["residual"] is None else y + s["residual"].float()
        out = {"y": y.to(getattr(torch, c["out"]))}
        if c["save_c"]:
            out["c"] = z.to(torch.bfloat16)
        return out
    dz = _plain_dact(s["dy"].float(), None if s["c"] is None else s["c"].float(), c["act"])
    kind = getattr(torch, c["out"])
    if s["offsets"] is None:
        out = {"dx": (dz @ w).to(torch.bfloat16), "dw": (dz.t() @ x).to(kind)}
        if s["bias"] is not None:
            out["db"] = dz.sum(0)
        return out
    mine = mine[:, :, None]
    dzg, xg = torch.where(mine, dz[row], 0.0), torch.where(mine, x[row], 0.0)
    out = {"dx": torch.bmm(dzg, w)[group, at].to(torch.bfloat16),
           "dw": torch.bmm(dzg.transpose(1, 2).contiguous(), xg).to(kind)}
    if s["bias"] is not None:
        out["db"] = dzg.sum(1)
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if not own:
        return {"route": _plain_route, "exchange": _plain_exchange, "linear": _plain_linear}[c["op"]](s, c)
    import moe_grouped_block_amd as mg
    if c["op"] == "route":
        how = dict(score=c["score"], renormalise=c["renormalise"])
        ids, weights = mg.route(s["logits"], c["top_k"], bias=s["bias"], **how)
        out = {"ids": ids, "weights": weights}
        if c["grad"]:
            out["dlogits"] = mg.route_backward(s["logits"], ids, s["dweights"], **how)
        return out
    if c["op"] == "exchange":
        if c["way"] == "backward":
            plan = mg.SortPlan(num_experts=c["experts"], m_aligned=c["m_aligned"], padded_offsets=s["offsets"],
                               row_of=s["row_of"], slot_of=s["slot_of"])
            drows, dweights = mg.combine_backward(s["dy"], plan, rows=s["rows"], weights=s["weights"],
                                                  out=s["buffer"])
            return {"drows": drows, "dweights": dweights, "dx": mg.dispatch_backward(s["da"], plan)}
        plan = mg.sort_tokens(s["ids"], c["experts"], weights=s["weights"], m_aligned=c["m_aligned"])
        out = {"offsets": plan.padded_offsets, "row_of": plan.row_of, "slot_of": plan.slot_of, "prob": plan.prob}
        if c["way"] == "forward":
            out["a"] = mg.dispatch(s["x"], plan, out=s["buffer"])
            out["y"] = mg.combine(s["rows"], plan, weights=s["weights"], residual=s["residual"])
            return out
        codes, scales = mg.dispatch(s["x"], plan, dtype=c["fmt"], sf_layout="kplanes", out=(s["buffer"], s["scales"]))
        out["a"] = codes.view(torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.float8_e5m2)
        out["scales"] = scales.view(torch.float8_e8m0fnu)
        return out
    if c["way"] == "forward":
        y = mg.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], offsets=s["offsets"],
                      save_c=c["save_c"], dtype=c["out"])
        return {"y": y[0], "c": y[1]} if c["save_c"] else {"y": y}
    need = ("dx", "dw", "db") if s["bias"] is not None else ("dx", "dw")
    got = mg.linear_backward(s["dy"], s["x"], s["w"], c=s["c"], act=c["act"], offsets=s["offsets"], need=need,
                             dw_dtype=c["out"])
    return {name: t for name, t in zip(("dx", "dw", "db"), got) if t is not None}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(c):
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        size = 4 if c["dtype"] == "float32" else 2
        # the gradient is a call of its own: it reads the logits again and writes as much
        return {"bytes": t * e * size * (3 if c["grad"] else 1) + t * k * (20 if c["grad"] else 8),
                "flops": t * e * (8 if c["grad"] else 4)}
    if c["op"] == "exchange":
        t, k, h = c["tokens"], c["top_k"], c["width"]
        slots = t * k
        rows = slots + min(slots, c["experts"]) * (c["m_aligned"] - 1) // 2
        if c["way"] == "forward":
            return {"bytes": 2 * h * (t + rows + slots + 2 * t) + slots * 24 + rows * 8, "flops": 2 * slots * h}
        if c["way"] == "quantise":
            return {"bytes": 2 * h * t + rows * h * 33 // 32 + slots * 16 + rows * 8, "flops": 4 * t * h}
        return {"bytes": 2 * h * (t + rows + 2 * slots + t) + slots * 16 + rows * 4, "flops": 4 * slots * h}
    m, n, k, groups = c["rows"], c["n"], c["k"], max(1, c["experts"])
    n_out = n // 2 if c["act"] == "swiglu" else n
    size = 4 if c["out"] == "float32" else 2
    weights = min(groups, m) * n * k
    if c["way"] == "forward":
        moved = 2 * (m * k + weights) + m * n_out * size + (2 * m * n_out if c["residual"] else 0) \
            + (2 * m * n if c["save_c"] else 0) + (4 * groups * n if c["bias"] else 0)
        return {"bytes": moved, "flops": 2 * m * n * k}
    moved = 2 * (m * k + weights + m * n_out) + (2 * m * n if c["act"] != "none" else 0) + 2 * m * k \
        + size * groups * n * k + (4 * groups * n if c["bias"] else 0)
    return {"bytes": moved, "flops": 4 * m * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "route":
        return _exact_route(s, c)
    if c["op"] == "exchange":
        return _exact_exchange(s, c)
    return _exact_linear(s, c)


def _exact_route(s, c):
    x = s["logits"].cpu().double().numpy()
    t, e = x.shape
    with np.errstate(all="ignore"):
        finite = np.where(np.isneginf(x).all(1, keepdims=True), 0.0, x)
        if c["score"] == "softmax":
            ex = np.exp(finite - finite.max(1, keepdims=True))
            p = np.where(np.isneginf(x), 0.0, ex / ex.sum(1, keepdims=True))
        else:
            p = np.exp(-np.logaddexp(0.0, -x))
        left = p + s["bias"].cpu().double().numpy() if c["bias"] else x.copy()
        left = np.where(np.isneginf(x), -np.inf, left)
    ids = np.full((t, c["top_k"]), -1, np.int64)
    w = np.zeros((t, c["top_k"]))
    every = np.arange(t)
    for j in range(c["top_k"]):                                           # the largest that is left, lowest index first
        best = left.argmax(1)
        there = left[every, best] > -np.inf
        ids[there, j], w[there, j] = best[there], p[every, best][there]
        left[every, best] = -np.inf
    chosen = w.copy()
    if c["renormalise"]:
        total = chosen.sum(1, keepdims=True)
        w = np.divide(chosen, total, out=np.zeros_like(chosen), where=total > 0)
    out = {"ids": ids.astype(np.int32), "weights": w}
    if c["grad"]:
        # through the weights' own Jacobian: d w_i / d s_j, then d s_j / d logit
        g = np.where(ids >= 0, s["dweights"].cpu().double().numpy(), 0.0)
        ds = g
        if c["renormalise"]:
            ds = np.divide(g * total - (g * chosen).sum(1, keepdims=True), total * total, out=np.zeros_like(g),
                           where=total > 0) * (ids >= 0)
        full = np.zeros((t, e))
        np.add.at(full, (every[:, None], np.maximum(ids, 0)), ds)
        if c["score"] == "softmax":
            out["dlogits"] = p * full - p * (p * full).sum(1, keepdims=True)
        else:
            out["dlogits"] = full * p * (1.0 - p)
    return out


def _exact_exchange(s, c):
    t, k, h, e, ma, cap = c["tokens"], c["top_k"], c["width"], c["experts"], c["m_aligned"], _capacity(c)
    ids = s["ids"].cpu().numpy()
    weights = s["weights"].cpu().double().numpy().reshape(-1)
    lists = [[] for _ in range(e)]
    for slot, g in enumerate(ids.reshape(-1).tolist()):
        if 0 <= g < e:
            lists[g].append(slot)
    row_of, slot_of, ends, at = np.full(t * k, -1, np.int64), np.full(cap, -1, np.int64), [], 0
    for members in lists:
        for i, slot in enumerate(members):
            row_of[slot], slot_of[at + i] = at + i, slot
        at += -(-len(members) // ma) * ma
        ends.append(at)
    used = np.flatnonzero(slot_of >= 0)
    token = torch.from_numpy(slot_of[used] // k).to(DEV)
    used_d = torch.from_numpy(used).to(DEV)
    w_row = torch.from_numpy(weights[slot_of[used]]).to(DEV)

    def summed(rows, factor):
        """Sum of the rows of every token, in 64 bits."""
        y = torch.zeros(t, h, dtype=torch.float64, device=DEV)
        for j in range(k):
            slots = np.arange(t) * k + j
            here = np.flatnonzero(row_of[slots] >= 0)
            put = torch.from_numpy(here).to(DEV)
            take = torch.from_numpy(row_of[slots[here]]).to(DEV)
            f = torch.from_numpy(weights[slots[here]]).to(DEV)[:, None] if factor else 1.0
            y[put] += rows[take].double() * f
        return y

    if c["way"] == "backward":
        drows = torch.zeros(cap, h, dtype=torch.float64, device=DEV)
        drows[used_d] = s["dy"][token].double() * w_row[:, None]
        dw = torch.zeros(t * k, dtype=torch.float64, device=DEV)
        dw[torch.from_numpy(slot_of[used]).to(DEV)] = (s["dy"][token].double() * s["rows"][used_d].double()).sum(1)
        return {"drows": drows, "dweights": dw.reshape(t, k), "dx": summed(s["da"], False)}
    prob = np.zeros(cap)
    prob[used] = weights[slot_of[used]]
    out = {"offsets": np.array(ends, np.int32), "row_of": row_of.reshape(t, k).astype(np.int32),
           "slot_of": slot_of.astype(np.int32), "prob": prob}
    a = torch.zeros(cap, h, dtype=torch.float64, device=DEV)
    a[used_d] = s["x"][token].double()
    if c["way"] == "forward":
        return {**out, "a": a, "y": summed(s["rows"], True) + s["residual"].double()}
    bits, low, most = (3, -6, 448.0) if c["fmt"] == "e4m3" else (2, -14, 57344.0)
    v = a.reshape(cap, h // 32, 32)
    scale = torch.full((cap, h // 32), 2.0 ** -127, dtype=torch.float64, device=DEV)
    for power in range(-126, 128):                                        # the smallest power of two that is enough
        scale = torch.where(v.abs().amax(2) > scale * most, 2.0 ** power, scale)
    v = v / scale[:, :, None]
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    out["a"] = (torch.round(v / unit) * unit).reshape(cap, h)             # torch.round: ties to even
    out["scales"] = scale.reshape(cap, h // 128, 4).permute(1, 0, 2).contiguous()
    return out


def _exact_linear(s, c):
    m, n, k = c["rows"], c["n"], c["k"]
    ends = [m] if s["offsets"] is None else s["offsets"].cpu().tolist()
    w = s["w"] if s["w"].dim() == 3 else s["w"][None]
    bias = None if s["bias"] is None else s["bias"].reshape(len(ends), n).double()
    parts, dw, at = [], [], 0
    db = torch.zeros(len(ends), n, dtype=torch.float64, device=DEV)
    for g, end in enumerate(ends):
        x = s["x"][at:end].double()
        if c["way"] == "forward":
            z = x @ w[g].double().t()
            parts.append(z if bias is None else z + bias[g])
        else:
            d = s["dy"][at:end].double()
            if c["act"] != "none":
                z = s["c"][at:end].double()
                if c["act"] == "swiglu":
                    lin = torch.cat([z[:, i:i + 32] for i in range(0, n, 64)], 1)
                    gate = torch.cat([z[:, i + 32:i + 64] for i in range(0, n, 64)], 1)
                    sig = torch.sigmoid(gate)
                    dl, dg = d * gate * sig, d * lin * (sig + gate * sig * torch.sigmoid(-gate))
                    d = torch.empty_like(z)
                    for i in range(n // 64):
                        d[:, 64 * i:64 * i + 32] = dl[:, 32 * i:32 * i + 32]
                        d[:, 64 * i + 32:64 * i + 64] = dg[:, 32 * i:32 * i + 32]
                elif c["act"] == "srelu":
                    d = torch.where(z > 0, 2.0 * z * d, 0.0)
                else:
                    sig = torch.sigmoid(2.0 * GELU_C * (z + GELU_A * z ** 3))
                    d = d * (sig + z * sig * (1.0 - sig) * 2.0 * GELU_C * (1.0 + 3.0 * GELU_A * z ** 2))
            parts.append(d @ w[g].double())
            dw.append(d.t() @ x)
            db[g] = d.sum(0)
        at = end
    got = torch.cat(parts, 0)
    if c["way"] == "backward":
        out = {"dx": got, "dw": torch.stack(dw).reshape(s["w"].shape)}
        if bias is not None:
            out["db"] = db.reshape(s["bias"].shape)
        return out
    y = got
    if c["act"] == "swiglu":
        y = torch.cat([got[:, i:i + 32] * got[:, i + 32:i + 64] * torch.sigmoid(got[:, i + 32:i + 64])
                       for i in range(0, n, 64)], 1)
    elif c["act"] == "srelu":
        y = torch.where(got > 0, got * got, 0.0)
    elif c["act"] == "gelu":
        y = got * torch.sigmoid(2.0 * GELU_C * (got + GELU_A * got ** 3))
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "c": got} if c["save_c"] else {"y": y}
