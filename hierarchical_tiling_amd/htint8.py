"""ctypes binding of include/htint8.h: products in 8-bit integers with scales for each token and each
channel, and the quantisation of rows that feeds them, with argument marshalling only.  Tensors are
passed as torch tensors (or, for the product, device addresses); every buffer is the caller's.
"""
from __future__ import annotations

import ctypes
import struct

from . import htgemm
from .htgemm import ACTS, DTYPES, GEMM_ERR_INVALID_ARG, GemmError, _check
from .htscaled import _bytes, _here, _padded, pitch, type_code

FORMS = {"single": 0, "batch": 1, "rows": 2}
_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class gemm_int8_desc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("d_type", _i32), ("form", _i32),
                ("lda", _i64), ("ldb", _i64), ("ldc", _i64), ("ldd", _i64),
                ("has_c", _i32), ("has_bias", _i32), ("act", _i32), ("split_k", _i32), ("batch", _i64),
                ("a_stride_l", _i64), ("b_stride_l", _i64), ("c_stride_l", _i64), ("d_stride_l", _i64),
                ("a_scale_l", _i64), ("b_scale_l", _i64)]


class gemm_int8_args(ctypes.Structure):
    _fields_ = [("A", _vp), ("a_scale", _vp), ("B", _vp), ("b_scale", _vp), ("C", _vp), ("D", _vp),
                ("bias", _vp), ("offsets", _vp), ("alpha", _f32), ("beta", _f32), ("workspace", _vp)]


class gemm_int8_info(ctypes.Structure):
    _fields_ = [("bm", _i32), ("bn", _i32), ("waves", _i32), ("lds_bytes", _i32), ("split_k", _i32),
                ("grid", _i64), ("name", ctypes.c_char * 64)]


class quant_rows_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("gate", _vp), ("x_type", _i32), ("act", _i32), ("rows", _i64), ("cols", _i64),
                ("ldx", _i64), ("ldg", _i64), ("row_index", _vp), ("x_rows", _i64), ("index_div", _i32),
                ("pad", _i32), ("q", _vp), ("ldq", _i64), ("scale", _vp)]


EXPORTED = ["gemm_int8_create", "gemm_int8_workspace_size", "gemm_int8_run", "gemm_int8_get_info",
            "gemm_int8_destroy", "quant_rows"]
_lib = None


def lib():
    """The loaded library with these entry points' signatures set."""
    global _lib
    if _lib is None:
        L = htgemm.lib()
        P, i = ctypes.POINTER, ctypes.c_int
        for name, args in {
                "gemm_int8_create": [P(gemm_int8_desc), P(_vp)],
                "gemm_int8_workspace_size": [_vp, P(ctypes.c_size_t)],
                "gemm_int8_run": [_vp, _vp, _vp],
                "gemm_int8_get_info": [_vp, P(gemm_int8_info)],
                "gemm_int8_destroy": [_vp],
                "quant_rows": [_vp, _vp]}.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, i
        _lib = L
    return _lib


def make_desc(M, N, K, out="bf16", *, lda, ldb, ldd, ldc=0, bias=False, act="none", groups=None, batch=None,
              split_k=0, a_stride_l=0, b_stride_l=0, c_stride_l=0, d_stride_l=0, a_scale_l=0,
              b_scale_l=0) -> gemm_int8_desc:
    """out: the type of D, C and bias.  groups: None (one product, or `batch` of them) or "rows".
    ldc > 0: C is read when beta != 0."""
    d = gemm_int8_desc()
    d.M, d.N, d.K, d.d_type = M, N, K, DTYPES[out]
    d.lda, d.ldb, d.ldc, d.ldd = lda, ldb, ldc, ldd
    d.has_c, d.has_bias, d.act = int(ldc > 0), int(bias), ACTS[act]
    d.form = FORMS[groups or ("single" if batch is None else "batch")]
    d.split_k, d.batch = split_k, 1 if batch is None else batch
    d.a_stride_l, d.b_stride_l, d.c_stride_l, d.d_stride_l = a_stride_l, b_stride_l, c_stride_l, d_stride_l
    d.a_scale_l, d.b_scale_l = a_scale_l, b_scale_l
    return d


_KINDS = {}


def _kinds(d_type):
    """The types of a description's codes, scales, outputs (C and bias among them) and offsets."""
    if not _KINDS:
        import torch
        _KINDS.update({DTYPES[n]: ((torch.int8,), (torch.float32,), (t,), (torch.int32,)) for n, t in
                       (("bf16", torch.bfloat16), ("f16", torch.float16), ("f32", torch.float32))})
    return _KINDS[d_type]


def _extents(d):
    """How many values from the first on A, a_scale, B, b_scale, C, D, bias and offsets have to hold
    for a product of description d."""
    M, N, K, L = d.M, d.N, d.K, d.batch if d.form != FORMS["single"] else 1
    if M == 0 or N == 0:
        return (0,) * 8
    many = L - 1 if d.form == FORMS["batch"] else 0
    b_many = 0 if d.form == FORMS["single"] else L - 1
    return (many * d.a_stride_l + (M - 1) * d.lda + K if K else 0, many * d.a_scale_l + M if K else 0,
            b_many * d.b_stride_l + (N - 1) * d.ldb + K if K else 0, b_many * d.b_scale_l + N if K else 0,
            many * d.c_stride_l + (M - 1) * d.ldc + N if d.has_c else 0, many * d.d_stride_l + (M - 1) * d.ldd + N,
            N if d.has_bias else 0, L + 1 if d.form == FORMS["rows"] else 0)


def _address(t, kinds, n, dev, rows, cols, ld):
    """Address of a tensor on device dev whose type is one of `kinds` and whose memory has n values
    from the first on; an address (or None) as it is.  The memory is read as rows of `cols` values, ld
    apart: a matrix of these rows and columns, or a vector (rows = 1), that lies otherwise raises."""
    if t is None or t.__class__ is int:
        return t or 0
    whole = t.is_contiguous()
    ok = t.get_device() == dev and t.dtype in kinds and (
        (whole and t.numel() >= n) or _bytes(t) >= n * t.element_size())
    if ok and n and rows > 1:
        if t.dim() > 1 and t.shape[-1] == cols and t.shape[-2] == rows:
            step, one = t.stride()[-2:]
            ok = step == ld and (one == 1 or cols == 1)
    elif ok and n and not whole and cols > 1:
        # the innermost dimension that has several values
        ok = next((step for size, step in zip(reversed(t.shape), reversed(t.stride())) if size > 1), 1) == 1
    if not ok:
        raise GemmError(GEMM_ERR_INVALID_ARG, "gemm_int8_run")
    return t.data_ptr()


_ARGS = struct.Struct("@8P2fP")   # gemm_int8_args, filled by one call
assert _ARGS.size == ctypes.sizeof(gemm_int8_args)


class Int8Gemm:
    """RAII wrapper: a handle for one product's description.

    run() raises GemmError for tensors on another device than the current one, of another type than
    the description's (codes: int8), or whose memory ends before the product's does, for matrices of the
    product's rows and columns whose strides are not the description's, for scales, bias and offsets
    whose values are not neighbours, and for a workspace of fewer than workspace_bytes.  Device
    addresses are taken as they are.  C is looked at only when beta is not 0."""

    def __init__(self, desc: gemm_int8_desc):
        self.handle = None
        self.desc = desc
        h = _vp()
        _check(lib().gemm_int8_create(ctypes.byref(desc), ctypes.byref(h)), "gemm_int8_create")
        self.handle = h.value
        self._kinds = _kinds(desc.d_type)
        self._extents = _extents(desc)
        self._room = self.workspace_bytes

    @property
    def info(self) -> gemm_int8_info:
        info = gemm_int8_info()
        _check(lib().gemm_int8_get_info(self.handle, ctypes.byref(info)), "gemm_int8_get_info")
        return info

    @property
    def workspace_bytes(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().gemm_int8_workspace_size(self.handle, ctypes.byref(n)), "gemm_int8_workspace_size")
        return n.value

    def run(self, A, a_scale, B, b_scale, D, C=None, bias=None, offsets=None, alpha=1.0, beta=0.0, workspace=None,
            stream=None):
        dev, stream = _here(stream)
        codes, f32, out, i32 = self._kinds
        nA, nSA, nB, nSB, nC, nD, n_bias, n_offsets = self._extents
        try:
            # the usual tensors, whole and of the right type, in one expression: _address for each
            # takes a call a microsecond more
            usual = (A.get_device() == dev and A.dtype in codes and A.numel() >= nA and A.is_contiguous() and
                     B.get_device() == dev and B.dtype in codes and B.numel() >= nB and B.is_contiguous() and
                     D.get_device() == dev and D.dtype in out and D.numel() >= nD and D.is_contiguous() and
                     a_scale.get_device() == dev and a_scale.dtype in f32 and a_scale.numel() >= nSA and
                     a_scale.is_contiguous() and
                     b_scale.get_device() == dev and b_scale.dtype in f32 and b_scale.numel() >= nSB and
                     b_scale.is_contiguous())
        except AttributeError:      # an address or None
            usual = False
        if usual:
            A, a_scale, B, b_scale, D = A.data_ptr(), a_scale.data_ptr(), B.data_ptr(), b_scale.data_ptr(), D.data_ptr()
        else:
            d = self.desc
            A, a_scale = _address(A, codes, nA, dev, d.M, d.K, d.lda), _address(a_scale, f32, nSA, dev, 1, d.M, 0)
            B, b_scale = _address(B, codes, nB, dev, d.N, d.K, d.ldb), _address(b_scale, f32, nSB, dev, 1, d.N, 0)
            D = _address(D, out, nD, dev, d.M, d.N, d.ldd)
        if C is None or not beta:
            C = 0
        else:
            C = _address(C, out, nC, dev, self.desc.M, self.desc.N, self.desc.ldc)
        bias = 0 if bias is None else _address(bias, out, n_bias, dev, 1, n_bias, 0)
        offsets = 0 if offsets is None else _address(offsets, i32, n_offsets, dev, 1, n_offsets, 0)
        if workspace is None:
            workspace = 0
        elif workspace.__class__ is not int:
            if workspace.get_device() != dev or (self._room and not (
                    (workspace.numel() >= self._room and workspace.is_contiguous()) or _bytes(workspace) >= self._room)):
                raise GemmError(GEMM_ERR_INVALID_ARG, "gemm_int8_run")
            workspace = workspace.data_ptr()
        rc = _lib.gemm_int8_run(self.handle, _ARGS.pack(A, a_scale, B, b_scale, C, D, bias, offsets, alpha, beta, workspace),
                                stream)
        if rc:
            raise GemmError(rc, "gemm_int8_run")

    def close(self):
        if self.handle:
            _check(lib().gemm_int8_destroy(self.handle), "gemm_int8_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_QUANT = struct.Struct("@2P2i4qPq2iPqP")   # quant_rows_args
assert _QUANT.size == ctypes.sizeof(quant_rows_args)


def _types():
    global _i8, _i32t, _f32t
    import torch
    _i32t, _f32t = torch.int32, torch.float32
    _i8 = torch.int8      # (last: another thread looks at it)


_i8 = _i32t = _f32t = None


def quantize(x, q, scale, gate=None, act=None, row_index=None, index_div=1, pad=False, stream=None):
    """quant_rows of a matrix x with contiguous rows: int8 codes q (rows, cols) and a float32 scale
    (rows) for each row.  With gate (x's shape and type) the values are act(gate) * x; act is "silu"
    where none is given.  With row_index (int32) the result has a row for each of its values.  pad: the
    bytes between the rows of q up to a multiple of 16 are the caller's too (behind the last row as
    well) and are set to zero.  Shapes and types that do not fit each other, memory that ends before
    the padding does, and tensors on another device than the current one raise GemmError."""
    if _i8 is None:
        _types()
    dev, stream = _here(stream)
    if x.dim() != 2:
        raise GemmError(GEMM_ERR_INVALID_ARG, "quantize")
    x_rows, cols = x.shape
    rows, index, ldg, at, code = x_rows, 0, 0, 0, 0
    ok = gate is not None or act is None
    if row_index is not None:
        rows, index = row_index.numel(), row_index.data_ptr()
        ok = ok and row_index.dtype is _i32t and row_index.is_contiguous() and row_index.get_device() == dev
    if gate is not None:
        ok = ok and gate.shape == x.shape and gate.dtype is x.dtype and gate.get_device() == dev
        if ok:
            ldg, at, code = pitch(gate, x_rows, cols), gate.data_ptr(), ACTS["silu" if act is None else act]
            ok = ldg >= 0
    ok = (ok and q.dtype is _i8 and scale.dtype is _f32t and q.shape == (rows, cols) and scale.numel() == rows and
          0 < index_div < 1 << 31 and scale.is_contiguous() and x.get_device() == dev and q.get_device() == dev and
          scale.get_device() == dev)
    if ok:
        step = cols if x.is_contiguous() else pitch(x, x_rows, cols)
        # (of one padded row the stride says how far its padding may go)
        to = cols if not pad and q.is_contiguous() else pitch(q, rows, cols)
        ok = step >= 0 and to >= 0 and (not pad or _padded(q, (0, to), rows, cols))
    if not ok:
        raise GemmError(GEMM_ERR_INVALID_ARG, "quantize")
    rc = (_lib or lib()).quant_rows(_QUANT.pack(x.data_ptr(), at, type_code(x), code, rows, cols, step, ldg, index,
                                                x_rows, index_div, pad, q.data_ptr(), to, scale.data_ptr()), stream)
    if rc:
        raise GemmError(rc, "quant_rows")
