"""ctypes binding of include/htscaled.h: block-scaled e4m3 products and the quantisation that feeds
them, with argument marshalling only.  Tensors are passed as torch tensors (or, for the product,
device addresses); every buffer is the caller's.
"""
from __future__ import annotations

import ctypes

from . import htgemm
from .htgemm import ACTS, DTYPES, GEMM_ERR_INVALID_ARG, GemmError, _addr, _check
from .htgemm import _stream as _stream_of

FORMS = {"single": 0, "batch": 1, "rows": 2, "k": 3}
_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class gemm_scaled_desc(ctypes.Structure):
    _fields_ = [("M", _i64), ("N", _i64), ("K", _i64), ("d_type", _i32), ("b_block", _i32),
                ("lda", _i64), ("ldb", _i64), ("ldc", _i64), ("ldd", _i64),
                ("a_scale_m", _i64), ("a_scale_k", _i64), ("b_scale_n", _i64), ("b_scale_k", _i64),
                ("has_c", _i32), ("has_bias", _i32), ("act", _i32), ("has_row_scale", _i32),
                ("form", _i32), ("split_k", _i32), ("batch", _i64),
                ("a_stride_l", _i64), ("b_stride_l", _i64), ("c_stride_l", _i64), ("d_stride_l", _i64),
                ("a_scale_l", _i64), ("b_scale_l", _i64)]


class gemm_scaled_args(ctypes.Structure):
    _fields_ = [("A", _vp), ("a_scale", _vp), ("B", _vp), ("b_scale", _vp), ("C", _vp), ("D", _vp),
                ("bias", _vp), ("row_scale", _vp), ("offsets", _vp), ("alpha", _f32), ("beta", _f32),
                ("workspace", _vp)]


class gemm_scaled_info(ctypes.Structure):
    _fields_ = [("bm", _i32), ("bn", _i32), ("waves", _i32), ("lds_bytes", _i32), ("split_k", _i32),
                ("grid", _i64), ("name", ctypes.c_char * 64)]


class quant_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_type", _i32), ("block_rows", _i32), ("pow2", _i32), ("index_div", _i32),
                ("rows", _i64), ("cols", _i64), ("ldx", _i64), ("row_index", _vp), ("x_rows", _i64),
                ("q", _vp), ("ldq", _i64), ("scale", _vp), ("scale_r", _i64), ("scale_c", _i64),
                ("qt", _vp), ("ldqt", _i64), ("scale_t", _vp), ("scale_t_c", _i64), ("scale_t_r", _i64),
                ("pad", _i32)]


EXPORTED = ["gemm_scaled_create", "gemm_scaled_workspace_size", "gemm_scaled_run", "gemm_scaled_get_info",
            "gemm_scaled_destroy", "quant_blocks"]
_lib = None


def _here(s):
    """(current device, hipStream_t of `s` or of torch's current stream): by the shorter way to the
    raw handle, since these calls are made many times a layer."""
    global _raw_stream, _device
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()      # initialises the runtime if nothing has
        _raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    dev = _device()
    return dev, _raw_stream(dev) if s is None else _stream_of(s)


_raw_stream = _device = None


def _elsewhere(dev, *tensors):
    """Whether any of the tensors (None and addresses aside) is not on device `dev`: a kernel there
    could not reach it."""
    for t in tensors:
        if t is not None and t.__class__ is not int and t.get_device() != dev:
            return True
    return False


def lib():
    """The loaded library with these entry points' signatures set."""
    global _lib
    if _lib is None:
        L = htgemm.lib()
        P, i = ctypes.POINTER, ctypes.c_int
        for name, args in {
                "gemm_scaled_create": [P(gemm_scaled_desc), P(_vp)],
                "gemm_scaled_workspace_size": [_vp, P(ctypes.c_size_t)],
                "gemm_scaled_run": [_vp, P(gemm_scaled_args), _vp],
                "gemm_scaled_get_info": [_vp, P(gemm_scaled_info)],
                "gemm_scaled_destroy": [_vp],
                "quant_blocks": [P(quant_args), _vp]}.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, i
        _lib = L
    return _lib


def make_desc(M, N, K, out="bf16", *, lda, ldb, ldd, ldc=0, b_block=128, a_scale_strides, b_scale_strides,
              bias=False, act="none", row_scale=False, groups=None, batch=None, split_k=0,
              a_stride_l=0, b_stride_l=0, c_stride_l=0, d_stride_l=0, a_scale_l=0,
              b_scale_l=0) -> gemm_scaled_desc:
    """a_scale_strides = (per row, per block of k), b_scale_strides = (per b_block columns, per block
    of k).  groups: None (one product, or `batch` of them), "rows" or "k".  ldc > 0: C is read when
    beta != 0."""
    d = gemm_scaled_desc()
    d.M, d.N, d.K, d.d_type, d.b_block = M, N, K, DTYPES[out], b_block
    d.lda, d.ldb, d.ldc, d.ldd = lda, ldb, ldc, ldd
    d.a_scale_m, d.a_scale_k = a_scale_strides
    d.b_scale_n, d.b_scale_k = b_scale_strides
    d.has_c, d.has_bias, d.act, d.has_row_scale = int(ldc > 0), int(bias), ACTS[act], int(row_scale)
    d.form = FORMS[groups or ("single" if batch is None else "batch")]
    d.split_k, d.batch = split_k, 1 if batch is None else batch
    d.a_stride_l, d.b_stride_l, d.c_stride_l, d.d_stride_l = a_stride_l, b_stride_l, c_stride_l, d_stride_l
    d.a_scale_l, d.b_scale_l = a_scale_l, b_scale_l
    return d


class ScaledGemm:
    """RAII wrapper: a handle for one block-scaled product description."""

    def __init__(self, desc: gemm_scaled_desc):
        self.handle = None
        self.desc = desc
        h = _vp()
        _check(lib().gemm_scaled_create(ctypes.byref(desc), ctypes.byref(h)), "gemm_scaled_create")
        self.handle = h.value

    @property
    def info(self) -> gemm_scaled_info:
        info = gemm_scaled_info()
        _check(lib().gemm_scaled_get_info(self.handle, ctypes.byref(info)), "gemm_scaled_get_info")
        return info

    @property
    def workspace_bytes(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().gemm_scaled_workspace_size(self.handle, ctypes.byref(n)), "gemm_scaled_workspace_size")
        return n.value

    def run(self, A, a_scale, B, b_scale, D, C=None, bias=None, row_scale=None, offsets=None, alpha=1.0,
            beta=0.0, workspace=None, stream=None):
        a = gemm_scaled_args(_addr(A), _addr(a_scale), _addr(B), _addr(b_scale), None if C is None else _addr(C),
                             _addr(D), None if bias is None else _addr(bias),
                             None if row_scale is None else _addr(row_scale),
                             None if offsets is None else _addr(offsets), alpha, beta,
                             None if workspace is None else _addr(workspace))
        dev, stream = _here(stream)
        if _elsewhere(dev, A, a_scale, B, b_scale, C, D, bias, row_scale, offsets, workspace):
            raise GemmError(GEMM_ERR_INVALID_ARG, "gemm_scaled_run")
        rc = _lib.gemm_scaled_run(self.handle, ctypes.byref(a), stream)
        if rc:
            raise GemmError(rc, "gemm_scaled_run")

    def close(self):
        if self.handle:
            _check(lib().gemm_scaled_destroy(self.handle), "gemm_scaled_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_TYPE_CODES = {}


def type_code(t) -> int:
    """gemm_dtype of a float32, float16 or bfloat16 tensor, -1 of any other."""
    if not _TYPE_CODES:
        import torch
        _TYPE_CODES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    return _TYPE_CODES.get(t.dtype, -1)


def pitch(t, rows, cols):
    """Row stride of a rows x cols tensor with contiguous rows of their own; -1 of any other (rows
    that overlap, as an expanded tensor's do, among them)."""
    step, one = t.stride()
    if one != 1 and cols > 1:
        return -1
    return step if step >= cols else cols if rows <= 1 else -1


def _codes(t, rows, cols):
    """(address, row stride) of a rows x cols tensor of bytes with contiguous rows; None: another."""
    if t.shape != (rows, cols) or t.element_size() != 1:
        return None
    step = pitch(t, rows, cols)
    return None if step < 0 else (t.data_ptr(), step)


def _scale(t, rows, cols):
    """(address, strides) of a rows x cols float32 tensor; None: another."""
    if t.shape != (rows, cols) or _TYPE_CODES.get(t.dtype, -1) != 0:
        return None
    return (t.data_ptr(), *t.stride())


_NO_CODES, _NO_SCALE = (None, 0), (None, 0, 0)


def quantize(x, q=None, scale=None, qt=None, scale_t=None, block_rows=1, pow2=False, row_index=None,
             index_div=1, pad=False, stream=None):
    """quant_blocks of a matrix x with contiguous rows: q (rows, cols) and scale (rows / block_rows,
    cols / 128), qt (cols, rows) and scale_t (cols, rows / 128), each any float32 strides.  With
    row_index the result has a row for each of its values.  pad: the bytes between the rows of q and
    qt up to a multiple of 16 are the caller's too (behind the last row as well) and are set to
    zero, so that a product may count them in K.  Shapes that do not fit each other, and tensors on
    another device than the current one, raise GemmError."""
    code = type_code(x)
    ok = x.dim() == 2
    if ok:
        x_rows, cols = x.shape
        step = pitch(x, x_rows, cols)
        rows, index = x_rows, None
        if row_index is not None:
            rows, index = row_index.numel(), row_index.data_ptr()
            ok = row_index.element_size() == 4 and not row_index.is_floating_point() and row_index.is_contiguous()
        rb, cb = -(-rows // 128), -(-cols // 128)
        q_at = _NO_CODES if q is None else _codes(q, rows, cols)
        qt_at = _NO_CODES if qt is None else _codes(qt, cols, rows)
        s_at = _NO_SCALE if scale is None else _scale(scale, rows if block_rows == 1 else rb, cb)
        st_at = _NO_SCALE if scale_t is None else _scale(scale_t, cols, rb)
        ok = ok and step >= 0 and q_at and qt_at and s_at and st_at
    if not ok:
        raise GemmError(GEMM_ERR_INVALID_ARG, "quantize")
    a = quant_args(x.data_ptr(), code, block_rows, pow2, index_div, rows, cols, step, index,
                   x_rows, *q_at, *s_at, *qt_at, *st_at, pad)
    dev, stream = _here(stream)
    if _elsewhere(dev, x, q, scale, qt, scale_t, row_index):
        raise GemmError(GEMM_ERR_INVALID_ARG, "quantize")
    rc = (_lib or lib()).quant_blocks(ctypes.byref(a), stream)
    if rc:
        raise GemmError(rc, "quant_blocks")
