"""Layer operators of libmoegg on torch tensors: route, sort / dispatch /
combine, linear, each with its gradient.

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
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Any

import moe_grouped_block_amd as mg

__all__ = ["route", "route_backward", "SortPlan", "sort_tokens", "sort_rows", "dispatch", "dispatch_backward",
           "combine", "combine_backward", "unsort", "linear", "linear_backward"]

_NAMES = {"bfloat16": "bf16", "float32": "f32"}


def _torch():
    import torch
    return torch


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


def _want(t, name: str, dtypes, shape, device=None):
    """A dense CUDA tensor of one of `dtypes` and of `shape` (None: any size)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a torch tensor expected, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {' or '.join(str(d) for d in dtypes)} expected, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and s != w for s, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple('*' if w is None else w for w in shape)} expected, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor expected, got strides {t.stride()}")
    if device is None:
        if t.device.type != "cuda":
            raise ValueError(f"{name}: a tensor on the GPU expected, got one on {t.device}")
    elif t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other tensors are on {device}")
    return t


class _On:
    """The device and stream of one call: current inside the block, so that
    what is allocated there belongs to that stream."""

    def __init__(self, device, stream):
        torch = _torch()
        self.block = None
        if stream is None:
            if torch.cuda.current_device() != device.index:
                self.block = torch.cuda.device(device)
            self.handle = torch.cuda.current_stream(device).cuda_stream
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"stream of {stream.device}, the tensors are on {device}")
        self.handle = stream.cuda_stream
        self.block = contextlib.ExitStack()
        self.block.enter_context(torch.cuda.device(device))
        self.block.enter_context(torch.cuda.stream(stream))

    def __enter__(self):
        if self.block is not None:
            self.block.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.block is not None:
            self.block.__exit__(*exc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _done(status: int) -> None:
    if status != 0:
        raise mg.MoeggError(status, mg.moegg_last_error())


# ---- route -------------------------------------------------------------------

def _route_problem(logits, top_k, score, renormalise, scale):
    torch = _torch()
    _want(logits, "logits", (torch.float32, torch.bfloat16), (None, None))
    return mg.moegg_route_problem(num_tokens=logits.shape[0], num_experts=logits.shape[1], top_k=top_k,
                                  dtype=mg.DTYPES["bf16" if logits.dtype == torch.bfloat16 else "f32"],
                                  score=_code(mg.SCORES, score, "score"), renormalise=1 if renormalise else 0,
                                  scale=scale)


def route(logits, top_k: int, *, score: str = "softmax", bias=None, renormalise: bool = True, scale: float = 1.0,
          stream=None):
    """(ids int32 (T, top_k), weights fp32 (T, top_k)) of the router logits (T, E), fp32 or bf16."""
    torch = _torch()
    p = _route_problem(logits, top_k, score, renormalise, scale)
    dev = logits.device
    if bias is not None:
        _want(bias, "bias", (torch.float32,), (p.num_experts,), dev)
    if top_k < 0:
        raise ValueError(f"top_k={top_k} negative")
    with _On(dev, stream) as s:
        ids = torch.empty((p.num_tokens, top_k), dtype=torch.int32, device=dev)
        weights = torch.empty((p.num_tokens, top_k), dtype=torch.float32, device=dev)
        _done(mg._load().moegg_route(ctypes.byref(p), logits.data_ptr(), _ptr(bias), ids.data_ptr(),
                                     weights.data_ptr(), s))
    return ids, weights


def route_backward(logits, ids, dweights, *, score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                   stream=None):
    """Gradient (T, E) of the logits, in their type, from the gradient of route()'s weights."""
    torch = _torch()
    _want(ids, "ids", (torch.int32,), (None, None))
    p = _route_problem(logits, ids.shape[1], score, renormalise, scale)
    dev, shape = logits.device, (p.num_tokens, p.top_k)
    _want(ids, "ids", (torch.int32,), shape, dev)
    _want(dweights, "dweights", (torch.float32,), shape, dev)
    with _On(dev, stream) as s:
        dlogits = torch.empty_like(logits)
        _done(mg._load().moegg_route_backward(ctypes.byref(p), logits.data_ptr(), ids.data_ptr(),
                                              dweights.data_ptr(), dlogits.data_ptr(), s))
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
    p = mg.moegg_sort_problem(num_tokens=num_tokens, top_k=top_k, num_experts=num_experts, m_aligned=m_aligned)
    p.rows = mg._load().moegg_sort_rows(ctypes.byref(p))
    if p.rows < 0:      # an invalid problem: the call itself says why
        _done(mg._load().moegg_sort(ctypes.byref(p), *[None] * 7, 0, None))
    return p


def sort_rows(num_tokens: int, top_k: int, num_experts: int, m_aligned: int = 128) -> int:
    """Rows that any routing of the tokens fits into."""
    return _sort_problem(num_tokens, top_k, num_experts, m_aligned).rows


def sort_tokens(ids, num_experts: int, *, weights=None, m_aligned: int = 128, stream=None) -> SortPlan:
    """Sort the slots of ids (T, k) by expert; ids outside 0..num_experts-1 are dropped."""
    torch = _torch()
    _want(ids, "ids", (torch.int32,), (None, None))
    dev = ids.device
    if weights is not None:
        _want(weights, "weights", (torch.float32,), tuple(ids.shape), dev)
    p = _sort_problem(ids.shape[0], ids.shape[1], num_experts, m_aligned)
    lib = mg._load()
    need = lib.moegg_sort_workspace(ctypes.byref(p))
    with _On(dev, stream) as s:
        offsets = torch.empty(num_experts, dtype=torch.int32, device=dev)
        row_of = torch.empty_like(ids)
        slot_of = torch.empty(p.rows, dtype=torch.int32, device=dev)
        prob = None if weights is None else torch.empty(p.rows, dtype=torch.float32, device=dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _done(lib.moegg_sort(ctypes.byref(p), ids.data_ptr(), _ptr(weights), offsets.data_ptr(), row_of.data_ptr(),
                             slot_of.data_ptr(), _ptr(prob), _ptr(ws), need, s))
    return SortPlan(num_experts, m_aligned, offsets, row_of, slot_of, prob)


def _exchange_problem(plan: SortPlan, width: int, dtype: str, sf_layout, dev):
    torch = _torch()
    if not isinstance(plan, SortPlan):
        raise TypeError(f"plan: a SortPlan expected, got {type(plan).__name__}")
    _want(plan.row_of, "plan.row_of", (torch.int32,), (None, None), dev)
    _want(plan.slot_of, "plan.slot_of", (torch.int32,), (None,), dev)
    _want(plan.padded_offsets, "plan.padded_offsets", (torch.int32,), (plan.num_experts,), dev)
    if dtype not in ("bf16", "e4m3", "e5m2", "e2m1x2"):
        raise ValueError(f"dtype={dtype!r}: one of bf16, e4m3, e5m2, e2m1x2 expected")
    return mg.moegg_exchange_problem(num_tokens=plan.num_tokens, rows=plan.rows, top_k=plan.top_k,
                                     num_experts=plan.num_experts, width=width, dtype=mg.DTYPES[dtype],
                                     sf_layout=_code(mg.SF_LAYOUTS, sf_layout, "sf_layout"))


def _row_shapes(rows: int, width: int, dtype: str, sf_layout: str):
    """Shapes of the sorted rows and of their scales (None for bf16)."""
    if dtype == "bf16":
        return (rows, width), None
    codes = (rows, width // 2) if dtype == "e2m1x2" else (rows, width)
    return codes, ((width // 128, rows, 4) if sf_layout == "kplanes" else (rows, width // 32))


def _row_outputs(out, rows, width, dtype, sf_layout, dev):
    """The caller's `out` checked, or new tensors: (rows tensor, scales or None)."""
    torch = _torch()
    shape, sf_shape = _row_shapes(rows, width, dtype, sf_layout)
    kind = torch.bfloat16 if dtype == "bf16" else torch.uint8
    if out is None:
        return (torch.empty(shape, dtype=kind, device=dev),
                None if sf_shape is None else torch.empty(sf_shape, dtype=torch.uint8, device=dev))
    if sf_shape is None:
        return _want(out, "out", (kind,), shape, dev), None
    if not isinstance(out, (tuple, list)) or len(out) != 2:
        raise TypeError("out: a pair (codes, scales) expected for MX rows")
    return _want(out[0], "out[0]", (kind,), shape, dev), _want(out[1], "out[1]", (torch.uint8,), sf_shape, dev)


def dispatch(x, plan: SortPlan, *, dtype="bf16", sf_layout: str = "row_major", out=None, stream=None):
    """Rows of x (T, H) in the plan's order: bf16 (rows, H), or (codes, scales)
    of an MX type as moegg_run takes them.  `out`: write there (rows behind the
    last expert keep what they hold; in new tensors they are undefined)."""
    torch = _torch()
    dtype = _dtype_name(dtype)
    _want(x, "x", (torch.bfloat16,), (None, None))
    dev = x.device
    p = _exchange_problem(plan, x.shape[1], dtype, sf_layout, dev)
    _want(x, "x", (torch.bfloat16,), (plan.num_tokens, None), dev)
    with _On(dev, stream) as s:
        rows, sf = _row_outputs(out, plan.rows, p.width, dtype, sf_layout, dev)
        _done(mg._load().moegg_dispatch(ctypes.byref(p), x.data_ptr(), plan.row_of.data_ptr(), plan.slot_of.data_ptr(),
                                        plan.padded_offsets.data_ptr(), rows.data_ptr(), _ptr(sf), s))
    return rows if sf is None else (rows, sf)


def combine(rows, plan: SortPlan, *, weights=None, residual=None, out=None, stream=None):
    """y (T, H) = residual + sum over a token's rows, times weights (T, k)."""
    torch = _torch()
    _want(rows, "rows", (torch.bfloat16,), (None, None))
    dev = rows.device
    p = _exchange_problem(plan, rows.shape[1], "bf16", "row_major", dev)
    _want(rows, "rows", (torch.bfloat16,), (plan.rows, None), dev)
    shape = (plan.num_tokens, p.width)
    if weights is not None:
        _want(weights, "weights", (torch.float32,), (plan.num_tokens, plan.top_k), dev)
    if residual is not None:
        _want(residual, "residual", (torch.bfloat16,), shape, dev)
    if out is not None:
        _want(out, "out", (torch.bfloat16,), shape, dev)
    with _On(dev, stream) as s:
        y = torch.empty(shape, dtype=torch.bfloat16, device=dev) if out is None else out
        _done(mg._load().moegg_combine(ctypes.byref(p), rows.data_ptr(), plan.row_of.data_ptr(), _ptr(weights),
                                       _ptr(residual), y.data_ptr(), s))
    return y


def combine_backward(dy, plan: SortPlan, *, rows=None, weights=None, dtype="bf16", sf_layout: str = "row_major",
                     out=None, stream=None):
    """(drows, dweights) of combine(): drows in the plan's order, bf16 or
    (codes, scales) of an MX type; dweights (T, k), None unless `rows` (what
    combine() read) is given."""
    torch = _torch()
    dtype = _dtype_name(dtype)
    _want(dy, "dy", (torch.bfloat16,), (None, None))
    dev = dy.device
    p = _exchange_problem(plan, dy.shape[1], dtype, sf_layout, dev)
    _want(dy, "dy", (torch.bfloat16,), (plan.num_tokens, None), dev)
    slots = (plan.num_tokens, plan.top_k)
    if rows is not None:
        _want(rows, "rows", (torch.bfloat16,), (plan.rows, p.width), dev)
    if weights is not None:
        _want(weights, "weights", (torch.float32,), slots, dev)
    with _On(dev, stream) as s:
        drows, sf = _row_outputs(out, plan.rows, p.width, dtype, sf_layout, dev)
        dweights = None if rows is None else torch.empty(slots, dtype=torch.float32, device=dev)
        _done(mg._load().moegg_combine_backward(
            ctypes.byref(p), dy.data_ptr(), plan.row_of.data_ptr(), plan.slot_of.data_ptr(),
            plan.padded_offsets.data_ptr(), _ptr(rows), _ptr(weights), drows.data_ptr(), _ptr(sf), _ptr(dweights), s))
    return (drows if sf is None else (drows, sf)), dweights


def dispatch_backward(drows, plan: SortPlan, *, out=None, stream=None):
    """Gradient (T, H) of dispatch()'s x: the sum of a token's rows."""
    return combine(drows, plan, out=out, stream=stream)


def unsort(values, plan: SortPlan, *, stream=None):
    """Per-row fp32 numbers (rows) back as (T, k): moegg_run's dprob as the gradient of the weights."""
    torch = _torch()
    _want(values, "values", (torch.float32,), (plan.rows,))
    dev = values.device
    _want(plan.row_of, "plan.row_of", (torch.int32,), (None, None), dev)
    with _On(dev, stream) as s:
        out = torch.empty((plan.num_tokens, plan.top_k), dtype=torch.float32, device=dev)
        _done(mg._load().moegg_unsort(values.data_ptr(), plan.row_of.data_ptr(), out.data_ptr(), out.numel(),
                                      plan.rows, s))
    return out


# ---- linear ----------------------------------------------------------------------

_LINEAR_ACTS = ("none", "swiglu", "srelu", "gelu")


def _linear_problem(x, w, act, dtype, offsets):
    """The problem struct and the group count as a shape prefix of w, bias and their gradients."""
    torch = _torch()
    if act not in _LINEAR_ACTS:
        raise ValueError(f"act={act!r}: one of {_LINEAR_ACTS} expected")
    if dtype not in ("bf16", "f32"):
        raise ValueError(f"dtype={dtype!r}: bf16 or f32 expected")
    _want(x, "x", (torch.bfloat16,), (None, None))
    dev = x.device
    if offsets is None:
        _want(w, "w", (torch.bfloat16,), (None, x.shape[1]), dev)
        lead = ()
    else:
        _want(offsets, "offsets", (torch.int32,), (None,), dev)
        lead = (offsets.shape[0],)
        _want(w, "w", (torch.bfloat16,), (lead[0], None, x.shape[1]), dev)
    return mg.moegg_linear_problem(m=x.shape[0], n=w.shape[-2], k=x.shape[1], num_groups=lead[0] if lead else 1,
                                   act=mg.ACTS[act], dtype=mg.DTYPES[dtype]), lead


def _workspace(need: int, dev):
    """`need` bytes; none for an invalid problem (-1), which the call itself refuses."""
    return _torch().empty(need, dtype=_torch().uint8, device=dev) if need > 0 else None


def linear(x, w, *, bias=None, act: str = "none", residual=None, offsets=None, save_c: bool = False, dtype="bf16",
           out=None, stream=None):
    """y = act(x w^T + bias) + residual: x (M, K) bf16, w (N, K) bf16, or with
    ``offsets`` (L, int32 ends of the groups' rows) w (L, N, K) and bias
    (L, N).  ``dtype`` of y: bf16 or f32.  With ``save_c`` returns (y, c), c
    the bf16 pre-activation that linear_backward() takes."""
    torch = _torch()
    dtype = _dtype_name(dtype)
    p, lead = _linear_problem(x, w, act, dtype, offsets)
    dev = x.device
    shape = (p.m, p.n // 2 if act == "swiglu" else p.n)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    if bias is not None:
        _want(bias, "bias", (torch.float32,), (*lead, p.n), dev)
    if residual is not None:
        _want(residual, "residual", (torch.bfloat16,), shape, dev)
    if out is not None:
        _want(out, "out", (kind,), shape, dev)
    lib = mg._load()
    need = lib.moegg_linear_workspace(ctypes.byref(p))
    with _On(dev, stream) as s:
        ws = _workspace(need, dev)
        y = torch.empty(shape, dtype=kind, device=dev) if out is None else out
        c = torch.empty((p.m, p.n), dtype=torch.bfloat16, device=dev) if save_c else None
        a = mg.moegg_linear_args(x=x.data_ptr(), w=w.data_ptr(), bias=_ptr(bias), residual=_ptr(residual),
                                 offsets=_ptr(offsets), y=y.data_ptr(), c=_ptr(c), workspace=_ptr(ws),
                                 workspace_bytes=need)
        _done(lib.moegg_linear(ctypes.byref(p), ctypes.byref(a), s))
    return (y, c) if save_c else y


def linear_backward(dy, x, w, *, c=None, act: str = "none", offsets=None, need=("dx", "dw", "db"), dw_dtype="bf16",
                    stream=None):
    """(dx, dw, db) of linear(), None for those not in ``need``; c is what
    linear(save_c=True) returned (not needed for act "none")."""
    torch = _torch()
    dw_dtype = _dtype_name(dw_dtype)
    need = set(need)
    if not need or not need <= {"dx", "dw", "db"}:
        raise ValueError(f"need={sorted(need)}: some of dx, dw, db expected")
    p, lead = _linear_problem(x, w, act, dw_dtype, offsets)
    dev = x.device
    _want(dy, "dy", (torch.bfloat16,), (p.m, p.n // 2 if act == "swiglu" else p.n), dev)
    if c is not None:
        _want(c, "c", (torch.bfloat16,), (p.m, p.n), dev)
    elif act != "none":
        raise ValueError(f"act={act!r} needs c")
    lib = mg._load()
    want = ("dx" in need) | ("dw" in need) << 1 | ("db" in need) << 2
    size = lib.moegg_linear_backward_workspace(ctypes.byref(p), want)
    with _On(dev, stream) as s:
        ws = _workspace(size, dev)
        dx = torch.empty((p.m, p.k), dtype=torch.bfloat16, device=dev) if "dx" in need else None
        dw = torch.empty((*lead, p.n, p.k), dtype=torch.float32 if dw_dtype == "f32" else torch.bfloat16,
                         device=dev) if "dw" in need else None
        db = torch.empty((*lead, p.n), dtype=torch.float32, device=dev) if "db" in need else None
        a = mg.moegg_linear_args(x=x.data_ptr(), w=w.data_ptr(), offsets=_ptr(offsets), c=_ptr(c), dy=dy.data_ptr(),
                                 dx=_ptr(dx), dw=_ptr(dw), db=_ptr(db), workspace=_ptr(ws), workspace_bytes=size)
        _done(lib.moegg_linear_backward(ctypes.byref(p), ctypes.byref(a), s))
    return dx, dw, db
