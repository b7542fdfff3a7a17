"""Plain float64 implementations of the layer operators (route, sort,
dispatch, combine, linear) and their gradients, from the definitions in
include/moegg.h, on CPU tensors.  They share no code with the library.

Bounds come from the formats: rounding to bf16 is off by at most 2^-8 of the
value, to fp32 by 2^-24; a sum of n fp32 products in any order by at most
n 2^-24 of the sum of their magnitudes."""
import math

import numpy as np
import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24
INF = math.inf


# ---- route -------------------------------------------------------------------

def route(logits, top_k, score, bias=None, renormalise=True, scale=1.0):
    """(ids, weights, p, chosen mask) in float64; ids by k rounds of argmax."""
    x = logits.double().clamp(max=torch.finfo(torch.float32).max)
    ok = (x > -INF)                                     # NaN: false
    if score == "softmax":
        top = torch.where(ok, x, -INF).amax(1, keepdim=True)
        top = torch.where(top == -INF, 0.0, top)
        e = torch.where(x == -INF, 0.0, torch.exp(x - top))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
        if bias is not None:                            # the choice leaves NaN experts out
            ec = torch.where(ok, e, 0.0)
            pc = ec / ec.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.exp(-torch.logaddexp(torch.zeros_like(x), -x))
        pc = p
    key = x.clone() if bias is None else pc + bias.double()
    key = torch.where(ok & (key > -INF), key, -INF)
    t = x.shape[0]
    ids = torch.full((t, top_k), -1, dtype=torch.int64)
    for j in range(top_k):
        best = torch.from_numpy(np.argmax(key.numpy(), 1))          # first of equals: the lowest index
        there = key.gather(1, best[:, None])[:, 0] > -INF
        ids[:, j] = torch.where(there, best, -1)
        key.scatter_(1, best[:, None], -INF)
    return ids, weights_of(x, ids, p, score, renormalise, scale), p


def weights_of(x, ids, p, score, renormalise, scale):
    there = ids >= 0
    at = ids.clamp(min=0)
    if not renormalise:
        return torch.where(there, scale * p.gather(1, at), 0.0)
    l = torch.where(there, x.gather(1, at), -INF)       # noqa: E741
    logp = l if score == "softmax" else -torch.logaddexp(torch.zeros_like(l), -l)
    logp = torch.where(there, logp, -INF)
    top = logp.amax(1, keepdim=True)
    u = torch.where(there, torch.exp(logp - torch.where(top == -INF, 0.0, top)), 0.0)
    return scale * u / u.sum(1, keepdim=True).clamp(min=1e-300)


def route_backward(logits, ids, dweights, score, renormalise=True, scale=1.0):
    """dlogits by the weights' Jacobian, float64."""
    x = logits.double().clamp(max=torch.finfo(torch.float32).max)
    t, e = x.shape
    ids = torch.where((ids >= 0) & (ids < e), ids.long(), -1)
    there = ids >= 0
    g = torch.where(there, dweights.double(), 0.0)
    if score == "softmax":
        top = torch.where(x > -INF, x, -INF).amax(1, keepdim=True)
        ex = torch.where(x == -INF, 0.0, torch.exp(x - torch.where(top == -INF, 0.0, top)))
        p = ex / ex.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.exp(-torch.logaddexp(torch.zeros_like(x), -x))
    w = weights_of(x, ids, p, score, renormalise, scale)
    if renormalise:
        d = w * (g - ((g * w).sum(1, keepdim=True) / scale if scale else 0.0))
        if score == "sigmoid":
            d = d * (1.0 - p.gather(1, ids.clamp(min=0)))
        d = torch.where(there, d, 0.0)
        return torch.zeros(t, e, dtype=torch.float64).scatter_add_(1, ids.clamp(min=0), d)
    full = torch.zeros(t, e, dtype=torch.float64).scatter_add_(1, ids.clamp(min=0), scale * g)
    if score == "softmax":
        return p * (full - (full * p).sum(1, keepdim=True))
    chosen = torch.zeros(t, e).scatter_add_(1, ids.clamp(min=0), there.float()) > 0
    return torch.where(chosen, full * p * torch.exp(-torch.logaddexp(torch.zeros_like(x), x)), 0.0)


# ---- sort, dispatch, combine ---------------------------------------------------

def sort(ids, experts, m_aligned, rows):
    """(offsets, row_of, slot_of) by walking over the slots."""
    ids = ids.numpy()
    lists = [[] for _ in range(experts)]
    for slot, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts:
            lists[e].append(slot)
    row_of, slot_of = np.full(ids.size, -1, np.int64), np.full(rows, -1, np.int64)
    offsets, at = [], 0
    for members in lists:
        row_of[members] = at + np.arange(len(members))
        slot_of[at:at + len(members)] = members
        at += -(-len(members) // m_aligned) * m_aligned
        offsets.append(at)
    return torch.tensor(offsets), torch.from_numpy(row_of.reshape(ids.shape)), torch.from_numpy(slot_of)


def dispatch(x, slot_of, top_k):
    y = torch.zeros(slot_of.numel(), x.shape[1], dtype=torch.float64)
    used = slot_of >= 0
    y[used] = x.double()[slot_of[used] // top_k]
    return y


def combine(rows, row_of, weights=None, residual=None):
    """(y, magnitude): the sum, and the sum of the terms' magnitudes."""
    t, k = row_of.shape
    y, mag = torch.zeros(t, rows.shape[1], dtype=torch.float64), torch.zeros(t, rows.shape[1], dtype=torch.float64)
    for j in range(k):
        there = row_of[:, j] >= 0
        term = rows.double()[row_of[there, j].long()]
        if weights is not None:
            term = term * weights.double()[there, j][:, None]
        y[there] += term
        mag[there] += term.abs()
    if residual is not None:
        y, mag = y + residual.double(), mag + residual.double().abs()
    return y, mag


def mx_encode(v, fmt):
    """(codes, scale bytes) of (rows, H) float64 values, blocks of 32."""
    import synth
    most = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1x2": 6.0}[fmt]
    enc = {"e4m3": synth.encode_e4m3, "e5m2": synth.encode_e5m2, "e2m1x2": synth.encode_e2m1}[fmt]
    b = v.reshape(v.shape[0], -1, 32).numpy()
    bad = ~np.isfinite(b).all(2)
    amax = np.abs(np.where(np.isfinite(b), b, 0.0)).max(2)
    byte = np.zeros(amax.shape, np.int64)                # smallest power of two >= amax / most, from 2^-127
    while True:
        small = amax > most * np.exp2(byte - 127.0)
        if not small.any():
            break
        byte[small] += 1
    byte[bad] = 255
    scaled = np.where(bad[:, :, None], 0.0, b) / np.exp2(np.where(bad, 0, byte) - 127.0)[:, :, None]
    codes = enc(scaled.reshape(v.shape).astype(np.float32))
    if fmt == "e2m1x2" and codes.shape[1] == v.shape[1]:
        codes = codes[:, 0::2] | codes[:, 1::2] << 4
    return codes, byte.astype(np.uint8)


# ---- linear ----------------------------------------------------------------------

C, A = math.sqrt(2.0 / math.pi), 0.044715


def act(z, kind):
    if kind == "swiglu":
        v = z.reshape(z.shape[0], z.shape[1] // 64, 2, 32)
        return (v[:, :, 0] * v[:, :, 1] * torch.sigmoid(v[:, :, 1])).reshape(z.shape[0], z.shape[1] // 2)
    if kind == "srelu":
        return z.clamp(min=0.0) ** 2
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(C * (z + A * z ** 3)))
    return z


def dact(dy, z, kind):
    """dz = dy act'(z)."""
    if kind == "none":
        return dy
    z = z.clone().requires_grad_(True)
    act(z, kind).backward(dy)
    return z.grad


def spans(offsets, m):
    ends = [m] if offsets is None else offsets.tolist()
    at, out = 0, []
    for e in ends:
        out.append((at, e))
        at = e
    return out


def linear(x, w, bias=None, kind="none", residual=None, offsets=None):
    """(y, z, |x||w| + |bias|) in float64; rows behind the last group are NaN."""
    m, n = x.shape[0], w.shape[-2]
    w3 = w.reshape(-1, n, w.shape[-1]).double()
    z, mag = torch.full((m, n), math.nan, dtype=torch.float64), torch.zeros(m, n, dtype=torch.float64)
    for g, (b, e) in enumerate(spans(offsets, m)):
        z[b:e] = x[b:e].double() @ w3[g].t()
        mag[b:e] = x[b:e].double().abs() @ w3[g].abs().t()
        if bias is not None:
            v = bias.reshape(-1, n)[g].double()
            z[b:e] += v
            mag[b:e] += v.abs()
    y = act(z, kind)
    return (y if residual is None else y + residual.double()), z, mag


def linear_backward(dy, x, w, c=None, kind="none", offsets=None):
    """{"dx", "dw", "db"} and the bounds of their errors, float64."""
    m, n, k = x.shape[0], w.shape[-2], w.shape[-1]
    w3 = w.reshape(-1, n, k).double()
    dz = dact(dy.double(), None if c is None else c.double(), kind)
    # dz's evaluation: 16 roundings of the value itself; gelu' is a sum of terms
    # up to 1.2 whose 1 - s may be off by a rounding of 1 times up to 25, and
    # swiglu's terms are dy times x or g times a factor of at most 1.3 with up
    # to 24 roundings in it
    ev = dz.abs() * (0.0 if kind == "none" else 16 * F32)
    if kind == "gelu":
        ev = ev + dy.double().abs() * 64 * F32
    if kind == "swiglu":
        most = c.double().abs().reshape(m, -1, 2, 32).amax(2) * dy.double().abs().reshape(m, -1, 32)
        ev = ev + (most * 32 * F32)[:, :, None].expand(-1, -1, 2, -1).reshape(m, n)
    # without an activation dz is dy, else it is rounded to bf16 for the products
    off = ev + dz.abs() * (0.0 if kind == "none" else BF16)
    dx, dxb = torch.full((m, k), math.nan, dtype=torch.float64), torch.zeros(m, k, dtype=torch.float64)
    dw, dwb, db, dbb = [], [], [], []
    for g, (b, e) in enumerate(spans(offsets, m)):
        d, o, xs = dz[b:e], off[b:e], x[b:e].double()
        dx[b:e] = d @ w3[g]
        dxb[b:e] = (o + (n + 8) * F32 * d.abs()) @ w3[g].abs()
        dw.append(d.t() @ xs)
        dwb.append((o + (e - b + 8) * F32 * d.abs()).t() @ xs.abs())
        db.append(d.sum(0))
        dbb.append((ev[b:e] + (e - b + 8) * F32 * d.abs()).sum(0))
    dw, dwb = torch.stack(dw).reshape(w.shape), torch.stack(dwb).reshape(w.shape)
    lead = w.shape[:-1]
    return {"dx": (dx, dxb), "dw": (dw, dwb), "db": (torch.stack(db).reshape(lead), torch.stack(dbb).reshape(lead))}


def linear_bound(z, mag, k, kind, residual, out_eps):
    """Bound of the error of y = act(z) + residual, z's sum of k products being
    off by at most (k + 8) 2^-24 of the sum of their magnitudes."""
    y = act(z, kind) if residual is None else act(z, kind) + residual.double()
    d = (k + 8) * F32 * mag
    if kind == "swiglu":
        v, e = z.reshape(z.shape[0], -1, 2, 32), d.reshape(z.shape[0], -1, 2, 32)
        x, g, dx, dg = v[:, :, 0].abs(), v[:, :, 1].abs(), e[:, :, 0], e[:, :, 1]
        b = (dx * (g + dg) + 1.1 * dg * x + 8 * F32 * x * g).reshape(z.shape[0], -1)
    elif kind == "srelu":
        b = 2 * z.abs() * d + d * d + 2 * F32 * z * z
    elif kind == "gelu":
        b = 1.13 * d + 16 * F32 * z.abs()
    else:
        b = d
    extra = 0.0 if residual is None else F32 * (y.abs() + residual.double().abs())
    return b * (1 + out_eps) + out_eps * y.abs() + extra + 1e-38
