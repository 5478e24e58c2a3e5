"""Exports, choice and refusals of the products in 8-bit integers, their quantisation and the rows of a
routing, on the host (the device check is replaced by HTGEMM_FAKE_ARCH; pointers here are numbers that
nothing reads)."""
import ctypes

import pytest
import torch

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S
from test_int8_product import SHAPES
from test_scaled_boundary import declared

KERNELS = {"any_64x128", "any_128x128", "stream_16x32_w4", "stream_16x16_w8", "stream_32x32_w4", "stream_64x32_w4",
           "tile_64x128_w2x2", "tile_64x128_w2x2x2", "tile_128x128_w2x2", "tile_128x128_w2x2x2", "pingpong_256x256"}


@pytest.fixture(autouse=True)
def fake_gfx950(monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")


def test_every_declared_symbol_is_exported():
    names = declared("htint8.h")
    assert names == set(Q.EXPORTED)
    lib = ctypes.CDLL(H.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


def desc(**kw):
    base = dict(M=64, N=96, K=256, lda=256, ldb=256, ldd=96)
    base.update(kw)
    return Q.make_desc(**base)


def created(d):
    h = ctypes.c_void_p()
    rc = Q.lib().gemm_int8_create(ctypes.byref(d), ctypes.byref(h))
    assert (rc == 0) == bool(h.value)
    if rc == 0:
        assert Q.lib().gemm_int8_destroy(h) == 0
    return rc


def test_every_kernel_is_chosen_for_a_tested_shape():
    found = set()
    for M, N, K in SHAPES:
        for ld in (-(-K // 16) * 16, K + 1):
            found.add(Q.Int8Gemm(Q.make_desc(M, N, K, lda=ld, ldb=ld, ldd=N)).info.name.decode())
    assert found == KERNELS


@pytest.mark.parametrize("kw", [{}, {"out": "f32"}, {"out": "f16"}, {"batch": 4, "d_stride_l": 64 * 96},
                                {"groups": "rows", "batch": 5}, {"split_k": 64}, {"M": 0}, {"K": 0, "lda": 0, "ldb": 0},
                                {"ldc": 100}, {"K": 131071, "lda": 131072, "ldb": 131071}, {"lda": 1 << 40}])
def test_valid_descriptors(kw):
    assert created(desc(**kw)) == 0


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), 1), (dict(N=1 << 31, ldd=1 << 31), 1), (dict(K=131072, lda=131072, ldb=131072), 1), (dict(act=9), 1),
    (dict(form=3), 1), (dict(form=-1), 1), (dict(split_k=65), 1), (dict(split_k=-1), 1), (dict(batch=2), 1),
    (dict(form=1, batch=0, d_stride_l=64 * 96), 1), (dict(form=2, batch=0), 1), (dict(form=2, batch=65536), 1),
    (dict(form=2, batch=2, split_k=2), 1), (dict(form=1, batch=2, d_stride_l=0), 1), (dict(has_c=2), 1), (dict(has_bias=-1), 1),
    (dict(d_type=3), 2), (dict(lda=255), 3), (dict(ldb=255), 3), (dict(ldd=95), 3), (dict(has_c=1, ldc=95), 3),
    (dict(form=1, batch=2, d_stride_l=64 * 96, a_stride_l=-1), 3), (dict(form=2, batch=2, b_scale_l=-1), 3),
    (dict(form=1, batch=2, d_stride_l=-1), 3)])
def test_refused_descriptors(change, status):
    d = desc()
    for k, v in change.items():
        setattr(d, k, v)
    assert created(d) == status


def test_launches_of_too_many_threads():
    """2^30 rows of 1 to 2^27 columns' tiles: no kernel's launch has 2^32 threads or more."""
    big = (1 << 30) - 1
    assert created(desc(M=big, N=1, ldd=1)) == 0
    assert created(desc(M=big, N=1 << 20, ldd=1 << 20)) == 1
    assert created(desc(M=big, N=1 << 20, ldd=1 << 20, lda=257, ldb=257)) == 1


def run(change=None, **kw):
    h = Q.Int8Gemm(desc(**kw))
    a = Q.gemm_int8_args(A=4096, a_scale=4096, B=4096, b_scale=4096, D=4096, alpha=1.0)
    for k, v in (change or {}).items():
        setattr(a, k, v)
    rc = Q.lib().gemm_int8_run(h.handle, ctypes.byref(a), None)
    return rc


@pytest.mark.parametrize("kw,change,status", [
    ({}, dict(A=None), 1), ({}, dict(b_scale=None), 1), ({}, dict(D=None), 1), ({}, dict(bias=4096), 1),
    ({}, dict(offsets=4096), 1), ({}, dict(beta=1.0), 1), ({"ldc": 96}, dict(beta=1.0), 1), ({"bias": True}, {}, 1),
    ({"groups": "rows", "batch": 2}, {}, 1), ({"split_k": 2}, {}, 1), ({"split_k": 2}, dict(workspace=4097), 1),
    ({}, dict(D=4097), 4), ({"out": "f32"}, dict(D=4098), 4), ({}, dict(a_scale=4098), 4), ({}, dict(b_scale=4097), 4),
    ({"bias": True}, dict(bias=4097), 4), ({"groups": "rows", "batch": 2}, dict(offsets=4098), 4),
    ({"ldc": 96}, dict(beta=1.0, C=4097), 4)])
def test_refused_runs(kw, change, status):
    assert run(change, **kw) == status


def test_handles():
    L = Q.lib()
    assert L.gemm_int8_run(None, None, None) == 7 and L.gemm_int8_destroy(None) == 0
    assert L.gemm_int8_workspace_size(None, None) == 7 and L.gemm_int8_get_info(None, None) == 7
    h = Q.Int8Gemm(desc())
    assert L.gemm_int8_run(h.handle, None, None) == 1 and L.gemm_int8_get_info(h.handle, None) == 1
    h.close()
    h.close()
    assert Q.Int8Gemm(desc(M=0)).workspace_bytes == 0
    assert run(dict(A=None, B=None, a_scale=None, b_scale=None, D=None), M=0) == 0


def quant(**kw):
    a = Q.quant_rows_args(x=4096, x_type=0, rows=4, cols=8, ldx=8, index_div=1, q=4096, ldq=8, scale=4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return Q.lib().quant_rows(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(cols=(1 << 24) + 1, ldx=1 << 25, ldq=1 << 25), 1), (dict(pad=2), 1),
    (dict(index_div=0), 1), (dict(act=3), 1), (dict(gate=4096, ldg=8, act=4), 1), (dict(row_index=4096, x_rows=-1), 1),
    (dict(q=None), 1), (dict(scale=None), 1), (dict(x=None), 1), (dict(x=None, row_index=4096, x_rows=1), 1),
    (dict(x_type=3), 2), (dict(x_type=-1), 2), (dict(ldx=7), 3), (dict(ldq=7), 3), (dict(gate=4096, ldg=7), 3),
    (dict(x=4098), 4), (dict(scale=4098), 4), (dict(row_index=4098, x_rows=4), 4), (dict(gate=4098, ldg=8), 4),
    (dict(x_type=2, x=4097), 4)])
def test_refused_quantisation(kw, status):
    assert quant(**kw) == status


def test_quantisation_of_nothing():
    assert quant(rows=0, x=None, q=None, scale=None) == 0
    assert Q.lib().quant_rows(None, None) == 1


def args(kind, **kw):
    a = {"gather": R.gather_args(x=4096, type=0, topk=2, tokens=4, cols=8, ldx=8, order=4096, slot=4096, y=4096, rows=8, ldy=8),
         "combine": R.combine_args(y=4096, type=0, weight_type=0, rows=8, cols=8, ldy=8, slot=4096, weights=4096, out=4096,
                                   ld_out=8, tokens=4, topk=2),
         "combine_grad": R.combine_grad_args(d_out=4096, y=4096, type=0, weight_type=0, tokens=4, rows=8, cols=8, ld_out=8,
                                             ldy=8, order=4096, slot=4096, weights=4096, d_y=4096, ld_dy=8, d_weights=4096,
                                             topk=2)}[kind]
    for k, v in kw.items():
        setattr(a, k, v)
    return getattr(R.lib(), "route_" + kind)(ctypes.byref(a), None)


@pytest.mark.parametrize("kind", ["gather", "combine", "combine_grad"])
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(topk=0), 1), (dict(topk=65), 1),
    (dict(tokens=(1 << 23) + 1), 1), (dict(rows=(1 << 26) + 1), 1), (dict(cols=(1 << 24) + 1), 1), (dict(type=3), 2),
    (dict(slot=4098), 4), (dict(y=4098), 4), (dict(cols=9), 3)])
def test_refused_rows(kind, kw, status):
    assert args(kind, **kw) == status


@pytest.mark.parametrize("kind,kw,status", [
    ("gather", dict(x=None), 1), ("gather", dict(y=None), 1), ("gather", dict(order=None), 1), ("gather", dict(order=4097), 4),
    ("combine", dict(slot=None), 1), ("combine", dict(out=None), 1), ("combine", dict(y=None), 1),
    ("combine", dict(weight_type=3), 2), ("combine", dict(add=4096, ld_add=7), 3), ("combine", dict(add=4097, ld_add=8), 4),
    ("combine", dict(weight_type=2, weights=4097), 4), ("combine_grad", dict(order=None), 1),
    ("combine_grad", dict(slot=None), 1), ("combine_grad", dict(weights=None), 1), ("combine_grad", dict(y=None), 1),
    ("combine_grad", dict(d_y=None, d_weights=None), 1), ("combine_grad", dict(d_out=None), 1),
    ("combine_grad", dict(weight_type=4), 2), ("combine_grad", dict(ld_dy=7), 3), ("combine_grad", dict(d_weights=4098), 4)])
def test_refused_arguments_of_rows(kind, kw, status):
    assert args(kind, **kw) == status
    assert getattr(R.lib(), "route_" + kind)(None, None) == 1


# ---- the binding: shapes and types that do not fit, on the host ---------------------------------
i8 = dict(dtype=torch.int8)
i32 = dict(dtype=torch.int32)


def refused(call):
    with pytest.raises(H.GemmError) as e:
        call()
    assert e.value.status == H.GEMM_ERR_INVALID_ARG


@pytest.fixture()
def on_device_minus_one(monkeypatch):
    """Tensors of the host as those of the current device."""
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: -1)


def test_binding_refuses_tensors_of_the_product(on_device_minus_one):
    h = Q.Int8Gemm(desc(split_k=2, bias=True))
    good = dict(A=torch.zeros(64, 256, **i8), a_scale=torch.zeros(64), B=torch.zeros(96, 256, **i8), b_scale=torch.zeros(96),
                D=torch.zeros(64, 96, dtype=torch.bfloat16), bias=torch.zeros(96, dtype=torch.bfloat16),
                workspace=torch.zeros(h.workspace_bytes, dtype=torch.uint8))
    for name, bad in (("A", torch.zeros(63, 256, **i8)), ("A", torch.zeros(64, 256, dtype=torch.uint8)),
                      ("a_scale", torch.zeros(63)), ("a_scale", torch.zeros(64, dtype=torch.float64)),
                      ("B", torch.zeros(96, 255, **i8)), ("b_scale", torch.zeros(95)), ("D", torch.zeros(64, 96)),
                      ("D", torch.zeros(64, 95, dtype=torch.bfloat16)), ("bias", torch.zeros(95, dtype=torch.bfloat16)),
                      ("bias", torch.zeros(96)), ("workspace", torch.zeros(h.workspace_bytes - 1, dtype=torch.uint8))):
        refused(lambda: h.run(**{**good, name: bad}))


@pytest.mark.parametrize("bad", [
    dict(x=torch.zeros(4, 9)), dict(x=torch.zeros(4)), dict(q=torch.zeros(4, 8, dtype=torch.uint8)),
    dict(q=torch.zeros(3, 8, **i8)), dict(q=torch.zeros(1, 8, **i8).expand(4, 8)), dict(q=torch.zeros(8, 4, **i8).t()),
    dict(scale=torch.zeros(3)), dict(scale=torch.zeros(8)[::2]), dict(scale=torch.zeros(4, dtype=torch.float16)),
    dict(gate=torch.zeros(4, 7)), dict(gate=torch.zeros(4, 8, dtype=torch.float16)), dict(act="silu"),
    dict(row_index=torch.zeros(3, **i32)), dict(row_index=torch.zeros(4, dtype=torch.int64)), dict(pad=True)])
def test_binding_refuses_tensors_of_the_quantisation(bad, on_device_minus_one):
    # rows 16 bytes apart whose memory ends a byte before the padding of the last
    q = torch.zeros(4 * 16 - 1, **i8).as_strided((4, 8), (16, 1))
    refused(lambda: Q.quantize(**{**dict(x=torch.zeros(4, 8), q=q, scale=torch.zeros(4)), **bad}))


def rows_of(kind, **kw):
    x, y, order, slot = torch.zeros(4, 8), torch.zeros(9, 8), torch.zeros(9, **i32), torch.zeros(4, 2, **i32)
    if kind == "gather":
        R.gather(**{**dict(x=x, order=order, slot=slot, y=y), **kw})
    elif kind == "combine":
        R.combine(**{**dict(y=y, slot=slot, out=x, weights=torch.zeros(4, 2)), **kw})
    else:
        R.combine_grad(**{**dict(d_out=x, y=y, order=order, slot=slot, weights=torch.zeros(4, 2), d_y=torch.zeros(9, 8),
                                 d_weights=torch.zeros(4, 2)), **kw})


@pytest.mark.parametrize("kind,bad", [
    ("gather", dict(x=torch.zeros(5, 8))), ("gather", dict(y=torch.zeros(8, 8))), ("gather", dict(y=torch.zeros(9, 8).half())),
    ("gather", dict(y=torch.zeros(1, 8).expand(9, 8))), ("gather", dict(order=torch.zeros(9).long())),
    ("gather", dict(slot=torch.zeros(3, 2, **i32))), ("gather", dict(x=torch.zeros(8, 4).t())),
    ("combine", dict(out=torch.zeros(4, 7))), ("combine", dict(out=torch.zeros(4, 8).half())),
    ("combine", dict(weights=torch.zeros(4, 3))), ("combine", dict(weights=torch.zeros(2, 4).t())),
    ("combine", dict(add=torch.zeros(3, 8))), ("combine", dict(slot=torch.zeros(4, 2))),
    ("combine", dict(out=torch.zeros(1, 8).expand(4, 8))),
    ("combine_grad", dict(y=None)), ("combine_grad", dict(d_y=None, d_weights=None)),
    ("combine_grad", dict(y=torch.zeros(8, 8))), ("combine_grad", dict(d_y=torch.zeros(9, 9))),
    ("combine_grad", dict(d_weights=torch.zeros(4, 2).half())), ("combine_grad", dict(weights=torch.zeros(4, 1))),
    ("combine_grad", dict(order=torch.zeros(10, **i32))), ("combine_grad", dict(d_y=torch.zeros(1, 8).expand(9, 8)))])
def test_binding_refuses_tensors_of_rows(kind, bad, on_device_minus_one):
    refused(lambda: rows_of(kind, **bad))


class Elsewhere:
    """What a call reads of a torch stream on device 1."""
    device_index, cuda_stream = 1, 0


@pytest.mark.parametrize("kind", ["gather", "combine", "combine_grad", "product", "quantise"])
def test_streams_and_tensors_of_another_device(kind, monkeypatch):
    """The current device is 0 by what the binding asks, and the tensors' -1; nothing reaches the library."""
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: 0)
    h = Q.Int8Gemm(desc())

    def call(**kw):
        if kind == "product":
            h.run(torch.zeros(64, 256, **i8), torch.zeros(64), torch.zeros(96, 256, **i8), torch.zeros(96),
                  torch.zeros(64, 96, dtype=torch.bfloat16), **kw)
        elif kind == "quantise":
            Q.quantize(torch.zeros(4, 8), torch.zeros(4, 8, **i8), torch.zeros(4), **kw)
        else:
            rows_of(kind, **kw)

    refused(call)
    refused(lambda: call(stream=Elsewhere()))
