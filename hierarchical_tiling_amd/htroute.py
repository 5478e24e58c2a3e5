"""ctypes binding of include/htroute.h: expert counts, offsets and row order, and the balance loss
with its gradient, with argument marshalling only.  Every buffer is the caller's torch tensor, on
the current device; shapes and types that do not fit raise GemmError.
"""
from __future__ import annotations

import ctypes
import functools

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


EXPORTED = ["route_workspace_size", "route_experts", "balance_loss", "balance_grad"]
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
                "balance_grad": [P(balance_grad_args), _vp]}.items():
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
