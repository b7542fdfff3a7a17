"""Plain float64 implementations of the norm, the router with groups and rows
kept in 8 bits, from the definitions in include/moegg.h, on CPU tensors, with
bounds from the formats (see layer_ref)."""
import math

import numpy as np
import torch

from layer_ref import BF16, F32, mx_encode  # noqa: F401  (encode: tests take it from here)

INF = math.inf
Q_MAX = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1x2": 6.0}


# ---- norm ------------------------------------------------------------------------

def rms_norm(h, weight, eps):
    h = h.double()
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * weight.double()


# y's evaluation: half a rounding of the mean of squares in the root, the root's
# own unit (2^-23), the products by its power of two (exact), its factor and the
# weight: 0.5 + 2 + 2 roundings; 8 taken
Y_OFF = 8 * F32


def rms_norm_backward(dy, h, weight, eps, dh=None):
    """dx, dw and the bounds of their errors in fp32."""
    dy, h, w = dy.double(), h.double(), weight.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    x, g = h * r, dy * w
    m, most = (g * x).mean(1, keepdim=True), (g * x).abs().mean(1, keepdim=True)
    dx = r * (g - x * m)
    # g: a rounding; x: 5; m: a rounding of every g and 6 of its own; their
    # difference, r (3) and the sum with dh: below 32 of the terms' magnitudes
    bound = 32 * F32 * r * (g.abs() + x.abs() * most)
    if dh is not None:
        dx = dx + dh.double()
        bound = bound + 2 * F32 * dh.double().abs()
    # dw: fp32 products of x (5 roundings) and their sum in any order
    return dx, bound + 2 * F32 * dx.abs(), (dy * x).sum(0), (h.shape[0] + 16) * F32 * (dy * x).abs().sum(0)


# ---- route with groups --------------------------------------------------------------

def route_grouped(logits, top_k, groups, top_groups, best, score, bias=None):
    """ids by sorting, group by group and token by token."""
    x = logits.double().clamp(max=torch.finfo(torch.float32).max)
    t, e = x.shape
    ok = x > -INF                                       # NaN: false
    if score == "softmax":
        top = torch.where(ok, x, -INF).amax(1, keepdim=True)
        top = torch.where(top == -INF, 0.0, top)
        p = torch.where(ok, torch.exp(x - top), 0.0)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.exp(-torch.logaddexp(torch.zeros_like(x), -x))
    key = x if bias is None else p + bias.double()
    key = torch.where(ok & (key > -INF), key, -INF).numpy()
    base = key if bias is not None or best == 1 else torch.where(ok, p, -INF).numpy()
    ids, size = np.full((t, top_k), -1, np.int64), e // groups
    for i in range(t):
        scores = []
        for g in range(groups):
            members = sorted(base[i, g * size:(g + 1) * size].tolist(), reverse=True)[:best]
            members = [v for v in members if v > -INF]
            scores.append(sum(members[1:], members[0]) if members else -INF)
        chosen = sorted(range(groups), key=lambda g: (-scores[g], g))[:top_groups]
        experts = sorted(j for g in chosen for j in range(g * size, (g + 1) * size))
        order = sorted(experts, key=lambda j: (-key[i, j], j))[:top_k]
        for q, j in enumerate(order):
            if key[i, j] > -INF:
                ids[i, q] = j
    return torch.from_numpy(ids)


# ---- rows in 8 (4) bits ---------------------------------------------------------------

def decode(codes, byte, fmt):
    """Values (rows, H) of codes and row-major scale bytes, by the bits."""
    codes = torch.as_tensor(codes).long()
    if fmt == "e2m1x2":
        codes = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1)
        bits, expo, bias, mant, sign = 1, (codes & 7) >> 1, 1, (codes & 1).double() / 2, codes >> 3
    elif fmt == "e4m3":
        bits, expo, bias, mant, sign = 3, (codes & 127) >> 3, 7, (codes & 7).double() / 8, codes >> 7
    else:
        bits, expo, bias, mant, sign = 2, (codes & 127) >> 2, 15, (codes & 3).double() / 4, codes >> 7
    v = torch.where(expo > 0, (1.0 + mant) * torch.exp2((expo - bias).double()), mant * 2.0 ** (1 - bias))
    v = torch.where(sign > 0, -v, v)
    byte = torch.as_tensor(byte).double()
    return v * torch.where(byte == 255, math.nan, torch.exp2(byte - 127.0)).repeat_interleave(32, 1)


def rowmajor(sf, layout):
    return sf if layout == "row_major" else sf.permute(1, 0, 2).reshape(sf.shape[1], -1)


def check_mx(codes, sf, fmt, want, off):
    """Codes and row-major scale bytes of `want` (finite, float64), whose fp32
    values may be off by `off`: every scale byte is that of an amax in reach,
    every value the nearest of its grid to a number in reach."""
    rows, width = want.shape
    codes, sf = codes.cpu(), sf.cpu()
    blocks = (rows, width // 32, 32)
    lo = (want.abs() - off).clamp(min=0.0).reshape(blocks).amax(2)
    hi = (want.abs() + off).reshape(blocks).amax(2)

    def byte_of(amax):
        mant, expo = torch.frexp(amax / Q_MAX[fmt])     # mant in [0.5, 1)
        expo = torch.where(mant == 0.5, expo - 1, expo)
        return torch.where(amax == 0, 0, (expo + 127).clamp(min=0))
    assert ((sf >= byte_of(lo)) & (sf <= byte_of(hi))).all()
    got = decode(codes, sf, fmt)
    scale = torch.exp2(sf.double() - 127.0).repeat_interleave(32, 1)
    # half a step of the grid: relative where it is normal, of the lowest step below
    rel, low = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17), "e2m1x2": (0.25, 0.25)}[fmt]
    bad = (got - want).abs() > torch.maximum(rel * want.abs(), low * scale) + 1.25 * off
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    return got
