"""ctypes binding of include/htscaled.h: block-scaled e4m3 products and the quantisation that feeds
them, with argument marshalling only.  Tensors are passed as torch tensors (or, for the product,
device addresses); every buffer is the caller's.
"""
from __future__ import annotations

import ctypes
import struct

from . import htgemm
from .htgemm import ACTS, DTYPES, GEMM_ERR_INVALID_ARG, GemmError, _check
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
    raw handle, since these calls are made many times a layer.  A torch stream of another device
    raises: a kernel on it would not reach the tensors."""
    global _raw_stream, _device
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()      # initialises the runtime if nothing has
        _device = torch._C._cuda_getDevice           # (first: another thread looks at the other)
        _raw_stream = torch._C._cuda_getCurrentRawStream
    dev = _device()
    if s is None:
        return dev, _raw_stream(dev)
    if getattr(s, "device_index", dev) != dev:
        raise GemmError(GEMM_ERR_INVALID_ARG, "stream")
    return dev, _stream_of(s)


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
                "gemm_scaled_run": [_vp, _vp, _vp],
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


_KINDS = {}


def _kinds(d_type):
    """The types of a description's codes, scales, outputs (C and bias among them) and offsets."""
    if not _KINDS:
        import torch
        codes, f32, i32 = (torch.float8_e4m3fn, torch.uint8, torch.int8), (torch.float32,), (torch.int32,)
        _KINDS.update({DTYPES["bf16"]: (codes, f32, (torch.bfloat16,), i32), DTYPES["f32"]: (codes, f32, f32, i32)})
    return _KINDS[d_type]


def _extents(d):
    """How many values from the first on A, a_scale, B, b_scale, C, D, bias, row_scale and offsets have
    to hold for a product of description d."""
    M, N, K, L = d.M, d.N, d.K, d.batch if d.form != FORMS["single"] else 1
    if M == 0 or N == 0:
        return (0,) * 9
    form = d.form
    a_many = L - 1 if form == FORMS["batch"] else 0
    b_many = L - 1 if form in (FORMS["batch"], FORMS["rows"]) else 0
    d_many = L - 1 if form in (FORMS["batch"], FORMS["k"]) else 0
    kb, nb = -(-K // 128), -(-N // d.b_block)
    a = a_many * d.a_stride_l + (M - 1) * d.lda + K if K else 0
    b = b_many * d.b_stride_l + (N - 1) * d.ldb + K if K else 0
    a_scale = a_many * d.a_scale_l + (M - 1) * d.a_scale_m + (kb - 1) * d.a_scale_k + 1 if K else 0
    b_scale = b_many * d.b_scale_l + (nb - 1) * d.b_scale_n + (kb - 1) * d.b_scale_k + 1 if K else 0
    c = d_many * d.c_stride_l + (M - 1) * d.ldc + N if d.has_c else 0
    return (a, a_scale, b, b_scale, c, d_many * d.d_stride_l + (M - 1) * d.ldd + N, N if d.has_bias else 0,
            M if d.has_row_scale else 0, L + 1 if form in (FORMS["rows"], FORMS["k"]) else 0)


def _bytes(t):
    """Bytes of a tensor's memory from its first value on, whatever its shape."""
    size = t.element_size()
    return t.untyped_storage().nbytes() - t.storage_offset() * size


def _address(t, kinds, n, dev):
    """Address of a tensor on device dev whose type is one of `kinds` and whose memory has n values
    from the first on; an address (or None) as it is."""
    if t is None or t.__class__ is int:
        return t or 0
    if t.get_device() != dev or t.dtype not in kinds or not (
            (t.numel() >= n and t.is_contiguous()) or _bytes(t) >= n * t.element_size()):
        raise GemmError(GEMM_ERR_INVALID_ARG, "gemm_scaled_run")
    return t.data_ptr()


_ARGS = struct.Struct("@9P2fP")   # gemm_scaled_args, filled by one call
assert _ARGS.size == ctypes.sizeof(gemm_scaled_args)


class ScaledGemm:
    """RAII wrapper: a handle for one block-scaled product description.

    run() raises GemmError for tensors on another device than the current one, of another type than
    the description's (codes: uint8, int8 or float8_e4m3fn), or whose memory ends before the
    product's does, and for a workspace of fewer than workspace_bytes.  Device addresses are taken
    as they are.  C is looked at only when beta is not 0."""

    def __init__(self, desc: gemm_scaled_desc):
        self.handle = None
        self.desc = desc
        h = _vp()
        _check(lib().gemm_scaled_create(ctypes.byref(desc), ctypes.byref(h)), "gemm_scaled_create")
        self.handle = h.value
        self._kinds = _kinds(desc.d_type)
        self._extents = _extents(desc)
        self._room = self.workspace_bytes

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
        dev, stream = _here(stream)
        codes, f32, out, i32 = self._kinds
        nA, nSA, nB, nSB, nC, nD, n_bias, n_rows, n_offsets = self._extents
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
            A, a_scale = _address(A, codes, nA, dev), _address(a_scale, f32, nSA, dev)
            B, b_scale = _address(B, codes, nB, dev), _address(b_scale, f32, nSB, dev)
            D = _address(D, out, nD, dev)
        C = 0 if C is None or not beta else _address(C, out, nC, dev)
        bias = 0 if bias is None else _address(bias, out, n_bias, dev)
        row_scale = 0 if row_scale is None else _address(row_scale, f32, n_rows, dev)
        offsets = 0 if offsets is None else _address(offsets, i32, n_offsets, dev)
        if workspace is None:
            workspace = 0
        elif workspace.__class__ is not int:
            if workspace.get_device() != dev or (self._room and _bytes(workspace) < self._room):
                raise GemmError(GEMM_ERR_INVALID_ARG, "gemm_scaled_run")
            workspace = workspace.data_ptr()
        rc = _lib.gemm_scaled_run(self.handle, _ARGS.pack(A, a_scale, B, b_scale, C, D, bias, row_scale, offsets, alpha, beta,
                                                          workspace), stream)
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


def _padded(t, at, rows, cols):
    """Whether the memory of codes `t` at (address, row stride) goes on behind the last row to where
    padding it with zeros ends."""
    return rows == 0 or cols == 0 or _bytes(t) >= (rows - 1) * at[1] + min(at[1], -(-cols // 16) * 16)


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
    zero, so that a product may count them in K.  Shapes that do not fit each other, memory that ends
    before the padding does, and tensors on another device than the current one raise GemmError."""
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
        if ok and pad:
            ok = (q is None or _padded(q, q_at, rows, cols)) and (qt is None or _padded(qt, qt_at, cols, rows))
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
