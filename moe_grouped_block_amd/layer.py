"""Layer operators of libmoegg on torch tensors: rms_norm, route, sort /
dispatch / combine, linear, each with its gradient, and rows kept in 8 bits.

Like the rest of the binding this module marshals arguments and never
computes: it checks types, shapes, contiguity and devices, allocates the
outputs that the caller does not pass, and calls the C function of the same
name (include/moegg.h says what each computes).  A wrong argument raises
``ValueError`` or ``TypeError`` here or ``MoeggError`` with the library's
message, before anything is enqueued.

Every function runs on ``stream`` (default: the current stream of the
tensors' device); outputs and workspaces are allocated on that stream, and a
workspace is never shared between calls, so calls on several streams and
captured graphs do not meet in one.  Tensors made on another stream have to
be ready and kept alive as for any other kernel launch.

The functions stand outside autograd: results have no history, whether an
operand requires a gradient or not, and writing to an ``out`` is not noted
there.  Each operator's gradient is the function named after it (for a
``torch.autograd.Function``, what its ``backward`` calls).
"""
from __future__ import annotations

import contextlib
import operator
from dataclasses import dataclass
from typing import Any

import torch

import moe_grouped_block_amd as mg

__all__ = ["route", "route_backward", "SortPlan", "sort_tokens", "sort_rows", "dispatch", "dispatch_backward",
           "combine", "combine_backward", "unsort", "linear", "linear_backward", "rms_norm", "rms_norm_backward",
           "quantise", "dequantise"]

_NAMES = {"bfloat16": "bf16", "float32": "f32"}


def _dtype_name(d) -> str:
    """'bf16' / 'f32' / 'e4m3' / ... from a name or a torch dtype."""
    if not isinstance(d, str):
        d = str(d).replace("torch.", "")
    return _NAMES.get(d, d)


def _code(table: dict, name, what: str) -> int:
    try:
        return table[name]
    except (KeyError, TypeError):
        raise ValueError(f"{what}={name!r}: one of {sorted(k for k in table if isinstance(k, str))} expected") from None


def _refuse(t, name: str, dtypes, shape, device) -> None:
    """Say what is wrong with a tensor that is not a dense GPU tensor of one
    of `dtypes`, of `shape` (None: any size), on `device` (None: any GPU)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a torch tensor expected, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {' or '.join(str(d) for d in dtypes)} expected, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and s != w for s, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple('*' if w is None else w for w in shape)} expected, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor expected, got strides {t.stride()}")
    if not t.is_cuda:
        raise ValueError(f"{name}: a tensor on the GPU expected, got one on {t.device}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, the other tensors are on cuda:{device}")


def _lead(t, name: str, dtypes, dims: int) -> int:
    """Check the tensor that leads a call (dense, on a GPU, `dims` dimensions); its device."""
    try:
        if t.dtype in dtypes and t.is_cuda and t.dim() == dims and t.is_contiguous():
            return t.get_device()
    except AttributeError:
        pass
    _refuse(t, name, dtypes, (None,) * dims, None)
    raise ValueError(f"{name}: not a dense GPU tensor")


def _want(t, name: str, dtype, shape: tuple, device: int) -> int:
    """Check a tensor of exactly this type, shape and device; its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, (dtype,), shape, device)
    raise ValueError(f"{name}: not a dense tensor on cuda:{device}")


def _count(v, name: str) -> int:
    """A size given as a number, inside what the C structs hold."""
    v = operator.index(v)
    if not 0 <= v < 1 << 31:
        raise ValueError(f"{name}={v} outside 0..2^31-1")
    return v


def _fits(sizes: int) -> None:
    """Refuse tensors' sizes (or-ed together) that the C structs do not hold: a
    32-bit field would cut them without a word."""
    if sizes >> 31:
        raise ValueError("a tensor's size above 2^31-1")


class _Guard:
    """Makes a device and a stream other than the current ones current until
    close(), so that what a call allocates belongs to its stream."""

    def __init__(self, device: int, stream):
        self.blocks = contextlib.ExitStack()
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
            self.blocks.enter_context(torch.cuda.device(device))
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device.index != device:
            raise ValueError(f"stream of {stream.device}, the tensors are on cuda:{device}")
        self.handle = stream.cuda_stream
        self.blocks.enter_context(torch.cuda.device(device))
        self.blocks.enter_context(torch.cuda.stream(stream))

    def close(self):
        self.blocks.close()


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same without torch's wrappers around them (3 us of a small call's 10)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(device: int, stream):
    """(stream handle, guard to close or None) of a call on `stream` (None: the current one of `device`)."""
    if stream is None and _current_device() == device:
        return _current_stream(device), None
    guard = _Guard(device, stream)
    return guard.handle, guard


def _done(status: int) -> None:
    if status != 0:
        raise mg.MoeggError(status, mg.moegg_last_error())


# ---- route -------------------------------------------------------------------

def _route_problem(logits, top_k, score, renormalise, scale):
    """The problem struct (fields in the order of the C struct)."""
    rows, experts = logits.shape
    _fits(experts | top_k)
    return mg.moegg_route_problem(rows, experts, top_k, 3 if logits.dtype is torch.bfloat16 else 5,
                                  _code(mg.SCORES, score, "score"), 1 if renormalise else 0, scale)


def route(logits, top_k: int, *, score: str = "softmax", bias=None, renormalise: bool = True, scale: float = 1.0,
          num_groups: int = 1, top_groups: int = 1, group_best: int = 1, stream=None):
    """(ids int32 (T, top_k), weights fp32 (T, top_k)) of the router logits (T, E), fp32 or bf16.  With
    ``num_groups`` the experts come in that many groups of neighbours and only those of the ``top_groups``
    groups with the largest scores can be chosen; a group's score is the sum of its ``group_best`` (1 or 2)
    largest scores with bias.  The gradient is route_backward() either way."""
    dev = _lead(logits, "logits", (torch.float32, torch.bfloat16), 2)
    p = _route_problem(logits, _count(top_k, "top_k"), score, renormalise, scale)
    b = None if bias is None else _want(bias, "bias", torch.float32, (p.num_experts,), dev)
    g = None
    if num_groups != 1 or top_groups != 1 or group_best != 1:
        g = mg.moegg_route_groups(_count(num_groups, "num_groups"), _count(top_groups, "top_groups"),
                                  _count(group_best, "group_best"))
    s, guard = _on(dev, stream)
    try:
        ids = logits.new_empty((p.num_tokens, p.top_k), dtype=torch.int32)
        weights = logits.new_empty((p.num_tokens, p.top_k), dtype=torch.float32)
        if g is None:
            st = mg._load().moegg_route(p, logits.data_ptr(), b, ids.data_ptr(), weights.data_ptr(), s)
        else:
            st = mg._load().moegg_route_grouped(p, g, logits.data_ptr(), b, ids.data_ptr(), weights.data_ptr(), s)
        _done(st)
    finally:
        if guard is not None:
            guard.close()
    return ids, weights


def route_backward(logits, ids, dweights, *, score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                   stream=None):
    """Gradient (T, E) of the logits, in their type, from the gradient of route()'s weights."""
    dev = _lead(logits, "logits", (torch.float32, torch.bfloat16), 2)
    _lead(ids, "ids", (torch.int32,), 2)
    shape = (logits.shape[0], ids.shape[1])
    p = _route_problem(logits, shape[1], score, renormalise, scale)
    i = _want(ids, "ids", torch.int32, shape, dev)
    g = _want(dweights, "dweights", torch.float32, shape, dev)
    s, guard = _on(dev, stream)
    try:
        dlogits = torch.empty_like(logits)
        _done(mg._load().moegg_route_backward(p, logits.data_ptr(), i, g, dlogits.data_ptr(), s))
    finally:
        if guard is not None:
            guard.close()
    return dlogits


# ---- sort, dispatch, combine ---------------------------------------------------

@dataclass
class SortPlan:
    """Tokens sorted by expert: what sort_tokens() returns and dispatch(),
    combine() and their gradients take."""
    num_experts: int
    m_aligned: int
    padded_offsets: Any    # (L) int32, ends of the experts' padded rows
    row_of: Any            # (T, k) int32, -1: dropped
    slot_of: Any           # (rows) int32, -1: padding
    prob: Any = None       # (rows) fp32, the rows' weights (moegg_run's prob)

    @property
    def num_tokens(self) -> int:
        return self.row_of.shape[0]

    @property
    def top_k(self) -> int:
        return self.row_of.shape[1]

    @property
    def rows(self) -> int:
        """Rows of the sorted tensors: every routing fits; padded_offsets[-1] of them are in use."""
        return self.slot_of.shape[0]


def _sort_problem(num_tokens, top_k, num_experts, m_aligned):
    lib = mg._load()
    p = mg.moegg_sort_problem(num_tokens, top_k, _count(num_experts, "num_experts"), _count(m_aligned, "m_aligned"), 0)
    rows = lib.moegg_sort_rows(p)
    if rows < 0:      # an invalid problem: the call itself says why
        _done(lib.moegg_sort(p, *[None] * 7, 0, None))
    p.rows = rows
    return p


def sort_rows(num_tokens: int, top_k: int, num_experts: int, m_aligned: int = 128) -> int:
    """Rows that any routing of the tokens fits into."""
    return _sort_problem(_count(num_tokens, "num_tokens"), _count(top_k, "top_k"), num_experts, m_aligned).rows


def sort_tokens(ids, num_experts: int, *, weights=None, m_aligned: int = 128, stream=None) -> SortPlan:
    """Sort the slots of ids (T, k) by expert; ids outside 0..num_experts-1 are dropped."""
    dev = _lead(ids, "ids", (torch.int32,), 2)
    shape = ids.shape
    w = None if weights is None else _want(weights, "weights", torch.float32, shape, dev)
    _fits(shape[1])
    p = _sort_problem(shape[0], shape[1], num_experts, m_aligned)
    lib, rows = mg._load(), p.rows
    need = lib.moegg_sort_workspace(p)
    s, guard = _on(dev, stream)
    try:
        # one allocation for the plan's tensors
        slots = shape[0] * shape[1]
        sizes = (slots, num_experts, rows, rows) if w is not None else (slots, num_experts, rows)
        store = ids.new_empty(sum(sizes))
        row_of = store.as_strided(shape, (shape[1], 1))
        _, offsets, slot_of, *prob = torch.split_with_sizes(store, sizes)
        prob = prob[0].view(torch.float32) if prob else None
        ws = ids.new_empty(need, dtype=torch.uint8) if need else None
        _done(lib.moegg_sort(p, ids.data_ptr(), w, offsets.data_ptr(), row_of.data_ptr(), slot_of.data_ptr(),
                             None if prob is None else prob.data_ptr(), None if ws is None else ws.data_ptr(), need, s))
    finally:
        if guard is not None:
            guard.close()
    return SortPlan(num_experts, m_aligned, offsets, row_of, slot_of, prob)


def _plan_rows_of(plan: SortPlan, dev: int):
    """(num_tokens, top_k, address of row_of) of a plan, checked."""
    if not isinstance(plan, SortPlan):
        raise TypeError(f"plan: a SortPlan expected, got {type(plan).__name__}")
    t = plan.row_of
    if _lead(t, "plan.row_of", (torch.int32,), 2) != dev:
        _want(t, "plan.row_of", torch.int32, tuple(t.shape), dev)
    return (*t.shape, t.data_ptr())


def _plan_pointers(plan: SortPlan, dev: int):
    """(num_tokens, top_k, rows, addresses of row_of, slot_of and padded_offsets) of a plan, checked."""
    tokens, top_k, row_of = _plan_rows_of(plan, dev)
    t = plan.slot_of
    if _lead(t, "plan.slot_of", (torch.int32,), 1) != dev:
        _want(t, "plan.slot_of", torch.int32, tuple(t.shape), dev)
    offsets = _want(plan.padded_offsets, "plan.padded_offsets", torch.int32, (_count(plan.num_experts, "num_experts"),), dev)
    return tokens, top_k, t.shape[0], row_of, t.data_ptr(), offsets


def _row_kind(dtype, sf_layout):
    """Name of the rows' type, its code and the layout's."""
    dtype = _dtype_name(dtype)
    if dtype not in ("bf16", "e4m3", "e5m2", "e2m1x2"):
        raise ValueError(f"dtype={dtype!r}: one of bf16, e4m3, e5m2, e2m1x2 expected")
    return dtype, mg.DTYPES[dtype], _code(mg.SF_LAYOUTS, sf_layout, "sf_layout")


def _row_outputs(out, like, rows: int, width: int, dtype: str, sf_layout: str, dev: int):
    """The caller's `out` checked, or new tensors: (rows tensor, its address, scales or None, their address)."""
    if dtype == "bf16":
        t = like.new_empty((rows, width)) if out is None else out
        return t, _want(t, "out", torch.bfloat16, (rows, width), dev), None, None
    shape = (rows, width // 2) if dtype == "e2m1x2" else (rows, width)
    sf_shape = (width // 128, rows, 4) if sf_layout == "kplanes" else (rows, width // 32)
    if out is None:
        out = like.new_empty(shape, dtype=torch.uint8), like.new_empty(sf_shape, dtype=torch.uint8)
    if not isinstance(out, (tuple, list)) or len(out) != 2:
        raise TypeError("out: a pair (codes, scales) expected for MX rows")
    return (out[0], _want(out[0], "out[0]", torch.uint8, shape, dev),
            out[1], _want(out[1], "out[1]", torch.uint8, sf_shape, dev))


def dispatch(x, plan: SortPlan, *, dtype="bf16", sf_layout: str = "row_major", out=None, stream=None):
    """Rows of x (T, H) in the plan's order: bf16 (rows, H), or (codes, scales)
    of an MX type as moegg_run takes them.  `out`: write there (rows behind the
    last expert keep what they hold; in new tensors they are undefined)."""
    dtype, kind, layout = _row_kind(dtype, sf_layout)
    dev = _lead(x, "x", (torch.bfloat16,), 2)
    tokens, top_k, rows, row_of, slot_of, offsets = _plan_pointers(plan, dev)
    width = x.shape[1]
    xp = _want(x, "x", torch.bfloat16, (tokens, width), dev)
    _fits(top_k | width)
    p = mg.moegg_exchange_problem(tokens, rows, top_k, plan.num_experts, width, kind, layout)
    s, guard = _on(dev, stream)
    try:
        t, tp, sf, sp = _row_outputs(out, x, rows, width, dtype, sf_layout, dev)
        _done(mg._load().moegg_dispatch(p, xp, row_of, slot_of, offsets, tp, sp, s))
    finally:
        if guard is not None:
            guard.close()
    return t if sf is None else (t, sf)


def combine(rows, plan: SortPlan, *, weights=None, residual=None, out=None, stream=None):
    """y (T, H) = residual + sum over a token's rows, times weights (T, k)."""
    bf16 = torch.bfloat16
    dev = _lead(rows, "rows", (bf16,), 2)
    tokens, top_k, row_of = _plan_rows_of(plan, dev)
    n_rows, width = plan.rows, rows.shape[1]
    rp = _want(rows, "rows", bf16, (n_rows, width), dev)
    shape = (tokens, width)
    w = None if weights is None else _want(weights, "weights", torch.float32, (tokens, top_k), dev)
    r = None if residual is None else _want(residual, "residual", bf16, shape, dev)
    _fits(top_k | width)
    p = mg.moegg_exchange_problem(tokens, n_rows, top_k, plan.num_experts, width, 3, 0)
    s, guard = _on(dev, stream)
    try:
        y = rows.new_empty(shape) if out is None else out
        _done(mg._load().moegg_combine(p, rp, row_of, w, r, _want(y, "out", bf16, shape, dev), s))
    finally:
        if guard is not None:
            guard.close()
    return y


def combine_backward(dy, plan: SortPlan, *, rows=None, weights=None, dtype="bf16", sf_layout: str = "row_major",
                     out=None, stream=None):
    """(drows, dweights) of combine(): drows in the plan's order, bf16 or
    (codes, scales) of an MX type; dweights (T, k), None unless `rows` (what
    combine() read) is given."""
    dtype, kind, layout = _row_kind(dtype, sf_layout)
    dev = _lead(dy, "dy", (torch.bfloat16,), 2)
    tokens, top_k, n_rows, row_of, slot_of, offsets = _plan_pointers(plan, dev)
    width = dy.shape[1]
    dp = _want(dy, "dy", torch.bfloat16, (tokens, width), dev)
    rp = None if rows is None else _want(rows, "rows", torch.bfloat16, (n_rows, width), dev)
    w = None if weights is None else _want(weights, "weights", torch.float32, (tokens, top_k), dev)
    _fits(top_k | width)
    p = mg.moegg_exchange_problem(tokens, n_rows, top_k, plan.num_experts, width, kind, layout)
    s, guard = _on(dev, stream)
    try:
        t, tp, sf, sp = _row_outputs(out, dy, n_rows, width, dtype, sf_layout, dev)
        dweights = None if rows is None else dy.new_empty((tokens, top_k), dtype=torch.float32)
        _done(mg._load().moegg_combine_backward(p, dp, row_of, slot_of, offsets, rp, w, tp, sp,
                                                None if dweights is None else dweights.data_ptr(), s))
    finally:
        if guard is not None:
            guard.close()
    return (t if sf is None else (t, sf)), dweights


def dispatch_backward(drows, plan: SortPlan, *, out=None, stream=None):
    """Gradient (T, H) of dispatch()'s x: the sum of a token's rows."""
    return combine(drows, plan, out=out, stream=stream)


def unsort(values, plan: SortPlan, *, stream=None):
    """Per-row fp32 numbers (rows) back as (T, k): moegg_run's dprob as the gradient of the weights."""
    dev = _lead(values, "values", (torch.float32,), 1)
    tokens, top_k, row_of = _plan_rows_of(plan, dev)
    rows = plan.rows
    vp = _want(values, "values", torch.float32, (rows,), dev)
    s, guard = _on(dev, stream)
    try:
        out = values.new_empty((tokens, top_k))
        _done(mg._load().moegg_unsort(vp, row_of, out.data_ptr(), tokens * top_k, rows, s))
    finally:
        if guard is not None:
            guard.close()
    return out


# ---- norm ------------------------------------------------------------------------

_STREAMS = (torch.bfloat16, torch.float32)
_TYPE_CODES = {torch.bfloat16: 3, torch.float32: 5}
_MX = {"e4m3": 1, "e2m1x2": 2, "e5m2": 4}


def _mx_kind(dtype, what: str):
    """Name and code of an MX type."""
    dtype = _dtype_name(dtype)
    return dtype, _code(_MX, dtype, what)


def rms_norm(x, weight, *, residual=None, h=None, eps: float = 1e-6, dtype="bf16", copy=None,
             sf_layout: str = "row_major", stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual
    (T, H), weight (H) fp32.  ``dtype`` of y: bf16, or an MX type as (codes,
    scales) that moegg_run takes; ``copy``: with a bf16 y, also the same in an
    MX type (what linear_backward() reads as x, or moegg_run as A).

    x is bf16 or fp32, the residual bf16 or fp32 (fp32 where x is); with one,
    the sum is returned last, in the residual's type: in ``h``, which may be
    the residual itself, or a new tensor.  Returns y, or a tuple of y, the
    copy and h as far as they were asked for."""
    dev = _lead(x, "x", _STREAMS, 2)
    shape = x.shape
    rows, width = shape
    _fits(width)
    wp = _want(weight, "weight", torch.float32, (width,), dev)
    kind, layout = x.dtype, _code(mg.SF_LAYOUTS, sf_layout, "sf_layout")
    code = stream_code = _TYPE_CODES[kind]
    rp = hp = yp = cp = sp = None
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in _STREAMS:
            _refuse(residual, "residual", _STREAMS, shape, dev)
        kind = residual.dtype
        stream_code = _TYPE_CODES[kind]
        rp = _want(residual, "residual", kind, shape, dev)
        hp = None if h is None else _want(h, "h", kind, shape, dev)
    elif h is not None:
        raise ValueError("h: the sum with a residual, and none was given")
    name, mx = _dtype_name(dtype), 0
    if name != "bf16":
        if copy is not None:
            raise ValueError("copy: for a bf16 y")
        name, mx = _mx_kind(name, "dtype")
    elif copy is not None:
        name, mx = _mx_kind(copy, "copy")
    p = mg.moegg_norm_problem(rows, width, code, stream_code, mx, layout, eps)
    s, guard = _on(dev, stream)
    try:
        out = []
        if copy is not None or not mx:
            y = torch.empty_like(x) if x.dtype is torch.bfloat16 else x.new_empty(shape, dtype=torch.bfloat16)
            yp = y.data_ptr()
            out.append(y)
        if mx:
            codes, cp, sf, sp = _row_outputs(None, x, rows, width, name, sf_layout, dev)
            out.append((codes, sf))
        if residual is not None:
            if hp is None:
                h = torch.empty_like(residual)
                hp = h.data_ptr()
            out.append(h)
        _done(mg._load().moegg_rms_norm(p, mg.moegg_norm_args(x.data_ptr(), rp, wp, hp, yp, cp, sp), s))
    finally:
        if guard is not None:
            guard.close()
    return out[0] if len(out) == 1 else tuple(out)


def rms_norm_backward(dy, h, weight, *, dh=None, eps: float = 1e-6, need=("dx", "dw"), stream=None):
    """(dx, dw) of rms_norm(), None for those not in ``need``: dy (T, H) bf16
    (an MX y's gradient is y's), h what rms_norm() returned (x where there was
    no residual), dh the gradient that reaches h from elsewhere (the residual
    stream), in h's type.  dx, in h's type and with dh included, is the gradient
    of x and of the residual alike."""
    need = set(need)
    if not need or not need <= {"dx", "dw"}:
        raise ValueError(f"need={sorted(need)}: some of dx, dw expected")
    dev = _lead(h, "h", _STREAMS, 2)
    rows, width = h.shape
    _fits(width)
    dp = _want(dy, "dy", torch.bfloat16, (rows, width), dev)
    wp = _want(weight, "weight", torch.float32, (width,), dev)
    gp = None if dh is None else _want(dh, "dh", h.dtype, (rows, width), dev)
    code = _TYPE_CODES[h.dtype]
    p = mg.moegg_norm_problem(rows, width, code, code, 0, 0, eps)
    lib = mg._load()
    size = lib.moegg_rms_norm_backward_workspace(p) if "dw" in need else 0     # -1: an invalid problem, which the call refuses
    s, guard = _on(dev, stream)
    try:
        dx = dw = dxp = dwp = wsp = None
        if "dx" in need:
            dx = torch.empty_like(h)
            dxp = dx.data_ptr()
        if "dw" in need:
            dw = torch.empty_like(weight)
            dwp = dw.data_ptr()
        if size > 0:
            ws = h.new_empty(size, dtype=torch.uint8)
            wsp = ws.data_ptr()
        a = mg.moegg_norm_args(None, None, wp, h.data_ptr(), None, None, None, dp, gp, dxp, dwp, wsp, size)
        _done(lib.moegg_rms_norm_backward(p, a, s))
    finally:
        if guard is not None:
            guard.close()
    return dx, dw


# ---- rows kept in 8 bits -------------------------------------------------------------

_KEPT = {"e4m3": 1, "e5m2": 4}
_KEPT_OR_NOT = {"bf16": 3, **_KEPT}


def _is_pair(t, name: str) -> None:
    if not isinstance(t, (tuple, list)) or len(t) != 2:
        raise TypeError(f"{name}: a pair (codes, scales) expected")


def _scales(t, name: str, rows: int, width: int, sf_layout: str, dev: int) -> int:
    """Address of the scales of rows kept in 8 bits (one of the pair's tensors)."""
    return _want(t, name, torch.uint8, (width // 128, rows, 4) if sf_layout == "kplanes" else (rows, width // 32), dev)


def quantise(x, *, dtype="e4m3", sf_layout: str = "row_major", out=None, stream=None):
    """(codes, scales) of x (T, H), bf16 or fp32, in 8 bits (e4m3 or e5m2): the
    rows that dispatch() and rms_norm() write and linear_backward() reads.
    ``out``: a pair to write to."""
    dev = _lead(x, "x", _STREAMS, 2)
    rows, width = x.shape
    _fits(width)
    dtype = _dtype_name(dtype)
    kind, layout = _code(_KEPT, dtype, "dtype"), _code(mg.SF_LAYOUTS, sf_layout, "sf_layout")
    s, guard = _on(dev, stream)
    try:
        codes, cp, sf, sp = _row_outputs(out, x, rows, width, dtype, sf_layout, dev)
        _done(mg._load().moegg_quantise(x.data_ptr(), _TYPE_CODES[x.dtype], rows, width, kind, layout, cp, sp, s))
    finally:
        if guard is not None:
            guard.close()
    return codes, sf


def dequantise(rows, *, dtype="e4m3", sf_layout: str = "row_major", to="bf16", stream=None):
    """x (T, H) in bf16 or fp32 (``to``) of its (codes, scales)."""
    _is_pair(rows, "rows")
    dev = _lead(rows[0], "rows[0]", (torch.uint8,), 2)
    n, width = rows[0].shape
    _fits(width)
    kind, layout = _code(_KEPT, _dtype_name(dtype), "dtype"), _code(mg.SF_LAYOUTS, sf_layout, "sf_layout")
    to = _dtype_name(to)
    code = _code(_LINEAR_DTYPES, to, "to")
    cp, sp = rows[0].data_ptr(), _scales(rows[1], "rows[1]", n, width, sf_layout, dev)
    s, guard = _on(dev, stream)
    try:
        x = rows[0].new_empty((n, width), dtype=torch.float32 if to == "f32" else torch.bfloat16)
        _done(mg._load().moegg_dequantise(cp, sp, n, width, kind, layout, x.data_ptr(), code, s))
    finally:
        if guard is not None:
            guard.close()
    return x


# ---- linear ----------------------------------------------------------------------

_LINEAR_ACTS = {"none": 0, "swiglu": 1, "srelu": 2, "gelu": 7}
_LINEAR_DTYPES = {"bf16": 3, "f32": 5}


def _linear_problem(x, w, act, dtype, offsets, x_dtype=torch.bfloat16):
    """(device, problem struct, leading shape of w, bias and their gradients, addresses of x, w and offsets)."""
    act_code, dtype_code = _code(_LINEAR_ACTS, act, "act"), _code(_LINEAR_DTYPES, dtype, "dtype")
    bf16 = torch.bfloat16
    dev = _lead(x, "x", (x_dtype,), 2)
    m, k = x.shape
    if offsets is None:
        _lead(w, "w", (bf16,), 2)
        n, groups, lead, op = w.shape[0], 1, (), None
    else:
        _lead(offsets, "offsets", (torch.int32,), 1)
        _lead(w, "w", (bf16,), 3)
        groups, n = offsets.shape[0], w.shape[1]
        lead, op = (groups,), _want(offsets, "offsets", torch.int32, (groups,), dev)
    wp = _want(w, "w", bf16, (*lead, n, k), dev)
    _fits(n | k | groups)
    return dev, mg.moegg_linear_problem(m, n, k, groups, act_code, dtype_code), lead, x.data_ptr(), wp, op


def linear(x, w, *, bias=None, act: str = "none", residual=None, offsets=None, save_c=False, dtype="bf16",
           out=None, stream=None):
    """y = act(x w^T + bias) + residual: x (M, K) bf16, w (N, K) bf16, or with
    ``offsets`` (L, int32 ends of the groups' rows) w (L, N, K) and bias
    (L, N).  ``dtype`` of y: bf16 or f32.  With ``save_c`` returns (y, c), c
    the pre-activation that linear_backward() takes: in bf16 (True or "bf16"), or
    kept in 8 bits ("e4m3" or "e5m2") as (codes, scales (M, N / 32)).  Rows behind the
    last group are not written: `out` keeps them, new tensors (c too) hold
    anything there."""
    dtype = _dtype_name(dtype)
    dev, p, lead, xp, wp, op = _linear_problem(x, w, act, dtype, offsets)
    m, n = p.m, p.n
    shape = (m, n // 2 if act == "swiglu" else n)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    bp = None if bias is None else _want(bias, "bias", torch.float32, (*lead, n), dev)
    rp = None if residual is None else _want(residual, "residual", torch.bfloat16, shape, dev)
    lib = mg._load()
    keep = None
    if isinstance(save_c, (str, torch.dtype)):
        kept = _code(_KEPT_OR_NOT, _dtype_name(save_c), "save_c")
        if kept != _KEPT_OR_NOT["bf16"]:
            keep = mg.moegg_linear_saved(3, 0, kept)
    # (-1: an invalid problem, which the call refuses)
    need = lib.moegg_linear_workspace(p) if keep is None else lib.moegg_linear_saving_workspace(p, keep)
    s, guard = _on(dev, stream)
    try:
        y = x.new_empty(shape, dtype=kind) if out is None else out
        yp = _want(y, "out", kind, shape, dev)
        c = sf = None
        if keep is not None:
            c, sf = x.new_empty((m, n), dtype=torch.uint8), x.new_empty((m, n // 32), dtype=torch.uint8)
            keep.c_sf = sf.data_ptr()
        elif save_c:
            c = x.new_empty((m, n))
        ws = x.new_empty(need, dtype=torch.uint8) if need > 0 else None
        a = mg.moegg_linear_args(xp, wp, bp, rp, op, yp, None if c is None else c.data_ptr(), None, None, None, None,
                                 None if ws is None else ws.data_ptr(), need)
        _done(lib.moegg_linear(p, a, s) if keep is None else lib.moegg_linear_saving(p, a, keep, s))
    finally:
        if guard is not None:
            guard.close()
    return (y, (c, sf)) if keep is not None else (y, c) if save_c else y


def linear_backward(dy, x, w, *, c=None, act: str = "none", offsets=None, need=("dx", "dw", "db"), dw_dtype="bf16",
                    x_dtype="bf16", c_dtype="bf16", sf_layout: str = "row_major", stream=None):
    """(dx, dw, db) of linear(), None for those not in ``need``; c is what
    linear(save_c=True) returned (not needed for act "none"), dy bf16 whatever
    linear()'s ``dtype`` was.  Rows of dx behind the last group hold anything.

    x and c may be kept in 8 bits, each as a pair (codes, scales) with its
    ``x_dtype`` / ``c_dtype`` ("e4m3" or "e5m2"): c what linear(save_c=...)
    returned, x what rms_norm(), dispatch() or quantise() wrote, with its scales
    in ``sf_layout``."""
    dw_dtype = _dtype_name(dw_dtype)
    need = set(need)
    if not need or not need <= {"dx", "dw", "db"}:
        raise ValueError(f"need={sorted(need)}: some of dx, dw, db expected")
    x_dtype, c_dtype = _dtype_name(x_dtype), _dtype_name(c_dtype)
    x8, c8 = x_dtype != "bf16", c is not None and c_dtype != "bf16"
    keep = None
    if x8 or c8:
        keep = mg.moegg_linear_saved(_code(_KEPT_OR_NOT, x_dtype, "x_dtype"), _code(mg.SF_LAYOUTS, sf_layout, "sf_layout"),
                                     _code(_KEPT_OR_NOT, c_dtype, "c_dtype") if c8 else 3)
    if x8:
        _is_pair(x, "x")
    dev, p, lead, xp, wp, op = _linear_problem(x[0] if x8 else x, w, act, dw_dtype, offsets,
                                               torch.uint8 if x8 else torch.bfloat16)
    m, n, k = p.m, p.n, p.k
    if x8:
        keep.x_sf = _scales(x[1], "x[1]", m, k, sf_layout, dev)
    dp = _want(dy, "dy", torch.bfloat16, (m, n // 2 if act == "swiglu" else n), dev)
    cp = None
    if c is not None and c8:
        _is_pair(c, "c")
        cp, keep.c_sf = _want(c[0], "c[0]", torch.uint8, (m, n), dev), _scales(c[1], "c[1]", m, n, "row_major", dev)
    elif c is not None:
        cp = _want(c, "c", torch.bfloat16, (m, n), dev)
    elif act != "none":
        raise ValueError(f"act={act!r} needs c")
    lib = mg._load()
    want = ("dx" in need) | ("dw" in need) << 1 | ("db" in need) << 2
    size = lib.moegg_linear_backward_workspace(p, want) if keep is None \
        else lib.moegg_linear_saved_backward_workspace(p, keep, want)
    s, guard = _on(dev, stream)
    try:
        dx = dw = db = dxp = dwp = dbp = wsp = None
        if size > 0:
            ws = w.new_empty(size, dtype=torch.uint8)
            wsp = ws.data_ptr()
        if want & 1:
            dx = w.new_empty((m, k)) if x8 else torch.empty_like(x)
            dxp = dx.data_ptr()
        if want & 2:
            dw = torch.empty_like(w, dtype=torch.float32) if dw_dtype == "f32" else torch.empty_like(w)
            dwp = dw.data_ptr()
        if want & 4:
            db = w.new_empty((*lead, n), dtype=torch.float32)
            dbp = db.data_ptr()
        a = mg.moegg_linear_args(xp, wp, None, None, op, None, cp, dp, dxp, dwp, dbp, wsp, size)
        _done(lib.moegg_linear_backward(p, a, s) if keep is None else lib.moegg_linear_saved_backward(p, a, keep, s))
    finally:
        if guard is not None:
            guard.close()
    return dx, dw, db
