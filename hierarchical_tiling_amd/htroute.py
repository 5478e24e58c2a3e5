"""ctypes binding of include/htroute.h: expert counts, offsets and row order, and the balance loss
with its gradient, with argument marshalling only.  Every buffer is the caller's torch tensor.
"""
from __future__ import annotations

import ctypes

from . import htgemm
from .htgemm import GEMM_ERR_INVALID_ARG, GemmError, _addr, _check, _stream
from .htscaled import type_code

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


def workspace_size(tokens, topk, experts) -> int:
    """Bytes of workspace that route() and balance_loss() need."""
    n = ctypes.c_size_t()
    _check(lib().route_workspace_size(tokens, topk, experts, ctypes.byref(n)), "route_workspace_size")
    return n.value


def _require(ok, what):
    if not ok:
        raise GemmError(GEMM_ERR_INVALID_ARG, what)


def _whole(t, dtype, n, what):
    """A contiguous tensor of `n` values of a type, or None."""
    _require(t is None or (t.dtype == dtype and t.numel() == n and t.is_contiguous()), what)


def _room(workspace, tokens, topk, experts, what):
    _require(workspace is not None and
             workspace.numel() * workspace.element_size() >= workspace_size(tokens, topk, experts), what)


def route(ids, counts, offsets, order=None, slot=None, mask=None, align=1, workspace=None, stream=None):
    """route_experts: ids (tokens, topk) int32 to counts (experts), offsets (experts + 1), order (at
    least tokens * topk + experts * (align - 1)) and slot (tokens, topk), all int32."""
    import torch
    what, i32 = "route", torch.int32
    _require(ids.dim() == 2 and ids.dtype == i32 and (ids.stride(1) == 1 or ids.shape[1] == 1), what)
    tokens, topk = ids.shape
    experts = counts.numel()
    _whole(counts, i32, experts, what)
    _whole(offsets, i32, experts + 1, what)
    _whole(slot, i32, tokens * topk, what)
    _whole(order, i32, 0 if order is None else order.numel(), what)
    _require(mask is None or (mask.element_size() == 1 and mask.numel() == tokens and mask.is_contiguous()), what)
    _room(workspace, tokens, topk, experts, what)
    a = route_args(ids.data_ptr(), _addr(mask), tokens, max(ids.stride(0), topk), topk, experts, align,
                   counts.data_ptr(), offsets.data_ptr(), _addr(order), 0 if order is None else order.numel(),
                   _addr(slot), workspace.data_ptr())
    _check(lib().route_experts(ctypes.byref(a), _stream(stream)), "route_experts")


def _logits(logits, counts, mask, what):
    import torch
    _require(logits.dim() == 2 and (logits.stride(1) == 1 or logits.shape[1] == 1), what)
    tokens, experts = logits.shape
    _whole(counts, torch.int32, experts, what)
    _require(mask is None or (mask.element_size() == 1 and mask.numel() == tokens and mask.is_contiguous()), what)
    return tokens, experts


def balance_loss(logits, counts, topk, loss, prob, live, mask=None, coef=1.0, workspace=None, stream=None):
    """balance_loss: logits (tokens, experts) and the routing's counts to loss (1), prob (experts)
    and live (1)."""
    import torch
    what = "balance_loss"
    tokens, experts = _logits(logits, counts, mask, what)
    _whole(loss, torch.float32, 1, what)
    _whole(prob, torch.float32, experts, what)
    _whole(live, torch.int32, 1, what)
    _room(workspace, tokens, topk, experts, what)
    a = balance_args(logits.data_ptr(), type_code(logits), experts, topk, coef, tokens,
                     max(logits.stride(0), experts), _addr(mask), counts.data_ptr(), loss.data_ptr(),
                     prob.data_ptr(), live.data_ptr(), workspace.data_ptr())
    _check(lib().balance_loss(ctypes.byref(a), _stream(stream)), "balance_loss")


def balance_grad(logits, counts, topk, live, d_loss, d_logits, mask=None, coef=1.0, stream=None):
    """balance_grad: the loss's gradient with respect to the logits, d_loss (1) times it, into
    d_logits (the logits' shape and type)."""
    import torch
    what = "balance_grad"
    tokens, experts = _logits(logits, counts, mask, what)
    _whole(live, torch.int32, 1, what)
    _whole(d_loss, torch.float32, 1, what)
    _require(d_logits.shape == logits.shape and d_logits.dtype == logits.dtype and
             (d_logits.stride(1) == 1 or experts == 1), what)
    a = balance_grad_args(logits.data_ptr(), type_code(logits), experts, topk, coef, tokens,
                          max(logits.stride(0), experts), _addr(mask), counts.data_ptr(), live.data_ptr(),
                          d_loss.data_ptr(), d_logits.data_ptr(), max(d_logits.stride(0), experts))
    _check(lib().balance_grad(ctypes.byref(a), _stream(stream)), "balance_grad")
