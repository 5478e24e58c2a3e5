"""ctypes binding of include/htroute.h: expert counts, offsets and row order, tokens to their experts'
rows and back, weighted, with the gradients, and the balance loss with its gradient, with argument
marshalling only.  Every buffer is the caller's torch tensor, on
the current device; shapes and types that do not fit raise GemmError.
"""
from __future__ import annotations

import ctypes
import functools
import struct

from . import htgemm
from .htgemm import GEMM_ERR_INVALID_ARG, GemmError, _check
from .htscaled import _elsewhere, _here, pitch, type_code

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class route_args(ctypes.Structure):
    _fields_ = [("ids", _vp), ("mask", _vp), ("tokens", _i64), ("ld_ids", _i64), ("topk", _i32),
                ("experts", _i32), ("align", _i32), ("counts", _vp), ("offsets", _vp), ("order", _vp),
                ("rows", _i64), ("slot", _vp), ("workspace", _vp)]


class balance_args(ctypes.Structure):
    _fields_ = [("logits", _vp), ("type", _i32), ("experts", _i32), ("topk", _i32), ("coef", _f32),
                ("tokens", _i64), ("ld", _i64), ("mask", _vp), ("counts", _vp), ("loss", _vp),
                ("prob", _vp), ("live", _vp), ("workspace", _vp)]


class balance_grad_args(ctypes.Structure):
    _fields_ = [("logits", _vp), ("type", _i32), ("experts", _i32), ("topk", _i32), ("coef", _f32),
                ("tokens", _i64), ("ld", _i64), ("mask", _vp), ("counts", _vp), ("live", _vp),
                ("d_loss", _vp), ("d_logits", _vp), ("ld_d", _i64)]


class gather_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("type", _i32), ("topk", _i32), ("tokens", _i64), ("cols", _i64), ("ldx", _i64),
                ("order", _vp), ("slot", _vp), ("y", _vp), ("rows", _i64), ("ldy", _i64)]


class combine_args(ctypes.Structure):
    _fields_ = [("y", _vp), ("type", _i32), ("weight_type", _i32), ("rows", _i64), ("cols", _i64), ("ldy", _i64),
                ("slot", _vp), ("weights", _vp), ("add", _vp), ("ld_add", _i64), ("out", _vp), ("ld_out", _i64),
                ("tokens", _i64), ("topk", _i32)]


class combine_grad_args(ctypes.Structure):
    _fields_ = [("d_out", _vp), ("y", _vp), ("type", _i32), ("weight_type", _i32), ("tokens", _i64), ("rows", _i64),
                ("cols", _i64), ("ld_out", _i64), ("ldy", _i64), ("order", _vp), ("slot", _vp), ("weights", _vp),
                ("d_y", _vp), ("ld_dy", _i64), ("d_weights", _vp), ("topk", _i32)]


# the same, filled by one call each
_GATHER = struct.Struct("@P2i3q3P2q")
_COMBINE = struct.Struct("@P2i3q3PqP2qi4x")
_COMBINE_GRAD = struct.Struct("@2P2i5q4PqPi4x")
assert _GATHER.size == ctypes.sizeof(gather_args) and _COMBINE.size == ctypes.sizeof(combine_args)
assert _COMBINE_GRAD.size == ctypes.sizeof(combine_grad_args)

MAX_TOPK = 64      # ROUTE_MAX_TOPK

EXPORTED = ["route_workspace_size", "route_experts", "balance_loss", "balance_grad", "route_gather", "route_combine",
            "route_combine_grad"]
_lib = None


def lib():
    """The loaded library with these entry points' signatures set."""
    global _lib
    if _lib is None:
        L = htgemm.lib()
        P = ctypes.POINTER
        for name, args in {
                "route_workspace_size": [_i64, _i32, _i32, P(ctypes.c_size_t)],
                "route_experts": [P(route_args), _vp],
                "balance_loss": [P(balance_args), _vp],
                "balance_grad": [P(balance_grad_args), _vp],
                "route_gather": [_vp, _vp], "route_combine": [_vp, _vp], "route_combine_grad": [_vp, _vp]}.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        _lib = L
    return _lib


def _bad(what):
    return GemmError(GEMM_ERR_INVALID_ARG, what)


def _is(t, dtype, n):
    """Whether t is a contiguous tensor of n values of a type."""
    return t.dtype is dtype and t.numel() == n and t.is_contiguous()


def _mask(mask, tokens, what):
    """Address of a mask of a byte for each token, or None."""
    if mask is None:
        return None
    if mask.element_size() != 1 or mask.numel() != tokens or not mask.is_contiguous():
        raise _bad(what)
    return mask.data_ptr()


@functools.lru_cache(maxsize=64)
def workspace_size(tokens, topk, experts) -> int:
    """Bytes of workspace that route() and balance_loss() need."""
    n = ctypes.c_size_t()
    _check(lib().route_workspace_size(tokens, topk, experts, ctypes.byref(n)), "route_workspace_size")
    return n.value


def _room(workspace, tokens, topk, experts, what):
    """Address of a workspace of the size these need."""
    if workspace is None or workspace.numel() * workspace.element_size() < workspace_size(tokens, topk, experts):
        raise _bad(what)
    return workspace.data_ptr()


def _types():
    global _i32t, _f32t
    import torch
    _f32t = torch.float32      # (first: another thread looks at the other)
    _i32t = torch.int32


_i32t = _f32t = None


def route(ids, counts, offsets, order=None, slot=None, mask=None, align=1, workspace=None, stream=None):
    """route_experts: ids (tokens, topk) int32 to counts (experts), offsets (experts + 1), order (at
    least tokens * topk + experts * (align - 1)) and slot (tokens, topk), all int32."""
    if _i32t is None:
        _types()
    if ids.dim() != 2 or ids.dtype is not _i32t:
        raise _bad("route")
    tokens, topk = ids.shape
    step = pitch(ids, tokens, topk)
    experts = counts.numel()
    rows = 0 if order is None else order.numel()
    if (step < 0 or not _is(counts, _i32t, experts) or not _is(offsets, _i32t, experts + 1) or
            (slot is not None and not _is(slot, _i32t, tokens * topk)) or
            (order is not None and not _is(order, _i32t, rows))):
        raise _bad("route")
    a = route_args(ids.data_ptr(), _mask(mask, tokens, "route"), tokens, step, topk, experts,
                   align, counts.data_ptr(), offsets.data_ptr(), None if order is None else order.data_ptr(), rows,
                   None if slot is None else slot.data_ptr(), _room(workspace, tokens, topk, experts, "route"))
    dev, stream = _here(stream)
    if _elsewhere(dev, ids, counts, offsets, order, slot, mask, workspace):
        raise _bad("route")
    rc = (_lib or lib()).route_experts(ctypes.byref(a), stream)
    if rc:
        raise GemmError(rc, "route_experts")


def _logits(logits, counts, what):
    if _i32t is None:
        _types()
    if logits.dim() != 2:
        raise _bad(what)
    tokens, experts = logits.shape
    step = pitch(logits, tokens, experts)
    if step < 0 or not _is(counts, _i32t, experts):
        raise _bad(what)
    return tokens, experts, step


def balance_loss(logits, counts, topk, loss, prob, live, mask=None, coef=1.0, workspace=None, stream=None):
    """balance_loss: logits (tokens, experts) and the routing's counts to loss (1), prob (experts)
    and live (1)."""
    tokens, experts, ld = _logits(logits, counts, "balance_loss")
    if not (_is(loss, _f32t, 1) and _is(prob, _f32t, experts) and _is(live, _i32t, 1)):
        raise _bad("balance_loss")
    a = balance_args(logits.data_ptr(), type_code(logits), experts, topk, coef, tokens, ld,
                     _mask(mask, tokens, "balance_loss"), counts.data_ptr(), loss.data_ptr(), prob.data_ptr(),
                     live.data_ptr(), _room(workspace, tokens, topk, experts, "balance_loss"))
    dev, stream = _here(stream)
    if _elsewhere(dev, logits, counts, loss, prob, live, mask, workspace):
        raise _bad("balance_loss")
    rc = (_lib or lib()).balance_loss(ctypes.byref(a), stream)
    if rc:
        raise GemmError(rc, "balance_loss")


def balance_grad(logits, counts, topk, live, d_loss, d_logits, mask=None, coef=1.0, stream=None):
    """balance_grad: the loss's gradient with respect to the logits, d_loss (1) times it, into
    d_logits (the logits' shape and type)."""
    tokens, experts, ld = _logits(logits, counts, "balance_grad")
    if d_logits.shape != logits.shape or d_logits.dtype is not logits.dtype:
        raise _bad("balance_grad")
    step = pitch(d_logits, tokens, experts)
    if step < 0 or not (_is(live, _i32t, 1) and _is(d_loss, _f32t, 1)):
        raise _bad("balance_grad")
    a = balance_grad_args(logits.data_ptr(), type_code(logits), experts, topk, coef, tokens, ld,
                          _mask(mask, tokens, "balance_grad"), counts.data_ptr(), live.data_ptr(), d_loss.data_ptr(),
                          d_logits.data_ptr(), step)
    dev, stream = _here(stream)
    if _elsewhere(dev, logits, counts, live, d_loss, d_logits, mask):
        raise _bad("balance_grad")
    rc = (_lib or lib()).balance_grad(ctypes.byref(a), stream)
    if rc:
        raise GemmError(rc, "balance_grad")


def gather(x, order, slot, y, stream=None, topk=None):
    """route_gather: the tokens x (tokens, cols) to their experts' rows y (rows, cols), by route()'s
    order (rows) and slot (tokens, topk); rows of no assignment become zeros.  slot may be None, with
    the number of assignments a token has as topk: the same rows, each token read once for every one.
    The gradient with respect to x is combine() of y's gradient without weights."""
    if _i32t is None:
        _types()
    dev, stream = _here(stream)
    if x.dim() != 2:
        raise _bad("gather")
    (tokens, cols), rows, at = x.shape, order.numel(), 0
    if slot is not None:
        if (slot.dim() != 2 or slot.dtype is not _i32t or slot.shape[0] != tokens or not slot.is_contiguous() or
                slot.get_device() != dev or topk not in (None, slot.shape[1])):
            raise _bad("gather")
        topk, at = slot.shape[1], slot.data_ptr()
    elif topk.__class__ is not int or not 1 <= topk <= MAX_TOPK:
        raise _bad("gather")
    if (order.dtype is not _i32t or y.dtype is not x.dtype or y.shape != (rows, cols) or not order.is_contiguous() or
            x.get_device() != dev or order.get_device() != dev or y.get_device() != dev):
        raise _bad("gather")
    ldx = cols if x.is_contiguous() else pitch(x, tokens, cols)
    ldy = cols if y.is_contiguous() else pitch(y, rows, cols)
    if ldx < 0 or ldy < 0:
        raise _bad("gather")
    rc = (_lib or lib()).route_gather(_GATHER.pack(x.data_ptr(), type_code(x), topk, tokens, cols, ldx, order.data_ptr(),
                                                   at, y.data_ptr(), rows, ldy), stream)
    if rc:
        raise GemmError(rc, "route_gather")


def combine(y, slot, out, weights=None, add=None, stream=None):
    """route_combine: the rows y (rows, cols) back to their tokens, out (tokens, cols) = add + the sum
    of weights (tokens, topk; 1 where none are given) times y's rows at slot (tokens, topk).  out may
    be add."""
    if _i32t is None:
        _types()
    dev, stream = _here(stream)
    if y.dim() != 2 or slot.dim() != 2:
        raise _bad("combine")
    (rows, cols), (tokens, topk) = y.shape, slot.shape
    if (slot.dtype is not _i32t or not slot.is_contiguous() or out.dtype is not y.dtype or out.shape != (tokens, cols) or
            y.get_device() != dev or slot.get_device() != dev or out.get_device() != dev):
        raise _bad("combine")
    ldy = cols if y.is_contiguous() else pitch(y, rows, cols)
    ld_out = cols if out.is_contiguous() else pitch(out, tokens, cols)
    ld_add = at = w = w_type = 0
    if add is not None:
        if add.dtype is not y.dtype or add.shape != (tokens, cols) or add.get_device() != dev:
            raise _bad("combine")
        ld_add, at = pitch(add, tokens, cols), add.data_ptr()
    if weights is not None:
        if weights.shape != (tokens, topk) or not weights.is_contiguous() or weights.get_device() != dev:
            raise _bad("combine")
        w, w_type = weights.data_ptr(), type_code(weights)
    if ldy < 0 or ld_out < 0 or ld_add < 0:
        raise _bad("combine")
    rc = (_lib or lib()).route_combine(_COMBINE.pack(y.data_ptr(), type_code(y), w_type, rows, cols, ldy, slot.data_ptr(), w,
                                                     at, ld_add, out.data_ptr(), ld_out, tokens, topk), stream)
    if rc:
        raise GemmError(rc, "route_combine")


def combine_grad(d_out, y, order, slot, weights, d_y=None, d_weights=None, stream=None):
    """route_combine_grad: the gradients of a weighted combine() from d_out (tokens, cols): d_y (rows,
    cols) of its rows and d_weights (tokens, topk) of its weights, either of them None.  y is read for
    d_weights only, and may be None without it."""
    if _i32t is None:
        _types()
    dev, stream = _here(stream)
    if d_out.dim() != 2 or slot.dim() != 2 or (d_y is None and d_weights is None) or (y is None and d_weights is not None):
        raise _bad("combine_grad")
    (tokens, cols), (n, topk), rows, dtype = d_out.shape, slot.shape, order.numel(), d_out.dtype
    if (order.dtype is not _i32t or slot.dtype is not _i32t or n != tokens or not order.is_contiguous() or
            not slot.is_contiguous() or weights.shape != (tokens, topk) or not weights.is_contiguous() or
            d_out.get_device() != dev or order.get_device() != dev or slot.get_device() != dev or weights.get_device() != dev):
        raise _bad("combine_grad")
    ld_out = cols if d_out.is_contiguous() else pitch(d_out, tokens, cols)
    ldy = ld_dy = at = to = d_w = 0
    if y is not None:
        if y.dtype is not dtype or y.shape != (rows, cols) or y.get_device() != dev:
            raise _bad("combine_grad")
        ldy, at = cols if y.is_contiguous() else pitch(y, rows, cols), y.data_ptr()
    if d_y is not None:
        if d_y.dtype is not dtype or d_y.shape != (rows, cols) or d_y.get_device() != dev:
            raise _bad("combine_grad")
        ld_dy, to = cols if d_y.is_contiguous() else pitch(d_y, rows, cols), d_y.data_ptr()
    if d_weights is not None:
        if (d_weights.dtype is not weights.dtype or d_weights.shape != (tokens, topk) or not d_weights.is_contiguous() or
                d_weights.get_device() != dev):
            raise _bad("combine_grad")
        d_w = d_weights.data_ptr()
    if ld_out < 0 or ldy < 0 or ld_dy < 0:
        raise _bad("combine_grad")
    rc = (_lib or lib()).route_combine_grad(
        _COMBINE_GRAD.pack(d_out.data_ptr(), at, type_code(d_out), type_code(weights), tokens, rows, cols, ld_out, ldy,
                           order.data_ptr(), slot.data_ptr(), weights.data_ptr(), to, ld_dy, d_w, topk), stream)
    if rc:
        raise GemmError(rc, "route_combine_grad")
