"""Exports and refusals of the block-scaled products, the quantisation and the routing, on the host
(the device check is replaced by HTGEMM_FAKE_ARCH; pointers here are numbers that nothing reads)."""
import ctypes
import os
import re

import pytest

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared(header):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return set(re.findall(r"^int\s+(\w+)\s*\(", text, re.M))


@pytest.mark.parametrize("header,module", [("htscaled.h", S), ("htroute.h", R)])
def test_every_declared_symbol_is_exported(header, module):
    names = declared(header)
    assert names == set(module.EXPORTED)
    lib = ctypes.CDLL(H.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


@pytest.fixture(autouse=True)
def fake_gfx950(monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")


def desc(**kw):
    base = dict(M=64, N=96, K=256, lda=256, ldb=256, ldd=96, a_scale_strides=(1, 64), b_scale_strides=(2, 1))
    base.update(kw)
    return S.make_desc(**base)


def created(d):
    h = ctypes.c_void_p()
    rc = S.lib().gemm_scaled_create(ctypes.byref(d), ctypes.byref(h))
    assert (rc == 0) == bool(h.value)
    if rc == 0:
        assert S.lib().gemm_scaled_destroy(h) == 0
    return rc


@pytest.mark.parametrize("kw", [{}, {"b_block": 1}, {"out": "f32"}, {"batch": 4, "d_stride_l": 64 * 96},
                                {"groups": "rows", "batch": 5}, {"groups": "k", "batch": 2, "d_stride_l": 64 * 96},
                                {"split_k": 64}, {"M": 0}, {"K": 0, "lda": 0, "ldb": 0}, {"ldc": 100}])
def test_valid_descriptors(kw):
    assert created(desc(**kw)) == 0


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), 1), (dict(K=1 << 31, lda=1 << 31, ldb=1 << 31), 1), (dict(b_block=64), 1), (dict(act=9), 1),
    (dict(form=4), 1), (dict(form=-1), 1), (dict(split_k=65), 1), (dict(split_k=-1), 1), (dict(batch=2), 1),
    (dict(form=1, batch=0, d_stride_l=64 * 96), 1), (dict(form=2, batch=0), 1), (dict(form=2, batch=65536), 1),
    (dict(form=2, batch=3, split_k=2), 1), (dict(form=1, batch=3), 1), (dict(form=3, batch=3), 1), (dict(has_bias=2), 1),
    (dict(d_type=1), 2), (dict(d_type=3), 2), (dict(lda=255), 3), (dict(ldb=255), 3), (dict(ldd=95), 3),
    (dict(has_c=1, ldc=95), 3), (dict(a_scale_m=-1), 3), (dict(b_scale_k=-1), 3),
    (dict(form=1, batch=2, d_stride_l=64 * 96, a_stride_l=-1), 3), (dict(form=2, batch=2, b_stride_l=-16), 3),
    (dict(form=3, batch=2, d_stride_l=-1), 3),
])
def test_refused_descriptors(change, status):
    d = desc()
    for k, v in change.items():
        setattr(d, k, v)
    assert created(d) == status


def test_null_and_dead_handles():
    L = S.lib()
    n, info = ctypes.c_size_t(), S.gemm_scaled_info()
    assert L.gemm_scaled_create(None, ctypes.byref(ctypes.c_void_p())) == 1
    assert L.gemm_scaled_create(ctypes.byref(desc()), None) == 1
    assert L.gemm_scaled_workspace_size(None, ctypes.byref(n)) == 7
    assert L.gemm_scaled_get_info(None, ctypes.byref(info)) == 7
    assert L.gemm_scaled_run(None, None, None) == 7
    assert L.gemm_scaled_destroy(None) == 0
    h = S.ScaledGemm(desc())
    assert L.gemm_scaled_run(h.handle, None, None) == 1
    assert L.gemm_scaled_workspace_size(h.handle, None) == 1


def test_another_device_is_refused(monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx942")
    assert created(desc()) == 5
    assert S.lib().quant_blocks(ctypes.byref(quant()), None) == 5
    assert R.lib().route_experts(ctypes.byref(route()), None) == 5
    assert R.lib().balance_loss(ctypes.byref(loss()), None) == 5
    assert R.lib().balance_grad(ctypes.byref(grad()), None) == 5


P = 1 << 20   # an aligned number in place of an address


def quant(**kw):
    a = S.quant_args(x=P, x_type=2, block_rows=1, pow2=0, index_div=1, rows=0, cols=256, ldx=256, q=P, ldq=256,
                     scale=P, scale_r=1, scale_c=1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    ({}, 0), (dict(rows=-1), 1), (dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 31), 1), (dict(block_rows=64), 1),
    (dict(pow2=2), 1), (dict(pad=2), 1), (dict(index_div=0), 1), (dict(rows=4, q=None), 1), (dict(rows=4, q=None, scale=None), 1),
    
    (dict(rows=4, scale=None), 1), (dict(rows=4, qt=P, ldqt=8), 1), (dict(rows=4, scale_t=P), 1),
    (dict(rows=4, block_rows=128, scale=None), 1), (dict(cols=0, x=None, q=None, scale=None), 0),
    (dict(rows=4, block_rows=128, qt=P, ldqt=4, scale_t=P), 1), (dict(row_index=P, x_rows=-1), 1), (dict(rows=2, x=None), 1),
    (dict(x_type=3), 2), (dict(x_type=7), 2), (dict(ldx=255), 3), (dict(ldq=255), 3), (dict(scale_r=-1), 3),
    (dict(rows=4, qt=P, ldqt=3, scale_t=P), 3), (dict(x=P + 1), 4), (dict(scale=P + 2), 4), (dict(row_index=P + 1), 4),
])
def test_quantise_refusals(change, status):
    assert S.lib().quant_blocks(ctypes.byref(quant(**change)), None) == status
    assert S.lib().quant_blocks(None, None) == 1


def route(**kw):
    a = R.route_args(ids=P, mask=None, tokens=4, ld_ids=2, topk=2, experts=8, align=16, counts=P, offsets=P, order=P,
                     rows=8 + 8 * 15, slot=P, workspace=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(topk=0), 1), (dict(topk=65, ld_ids=65), 1), (dict(experts=0), 1), (dict(experts=1025), 1),
    (dict(align=0), 1), (dict(align=1025), 1), (dict(tokens=1 << 30), 1), (dict(ids=None), 1), (dict(counts=None), 1),
    (dict(offsets=None), 1), (dict(workspace=None), 1), (dict(rows=8 + 8 * 15 - 1), 1), (dict(ld_ids=1), 3),
    (dict(ids=P + 1), 4), (dict(offsets=P + 2), 4), (dict(workspace=P + 8), 4),
])
def test_route_refusals(change, status):
    assert R.lib().route_experts(ctypes.byref(route(**change)), None) == status
    assert R.lib().route_experts(None, None) == 1


def loss(**kw):
    a = R.balance_args(logits=P, type=2, experts=8, topk=2, coef=1.0, tokens=4, ld=8, mask=None, counts=P, loss=P, prob=P,
                       live=P, workspace=P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def grad(**kw):
    a = R.balance_grad_args(logits=P, type=2, experts=8, topk=2, coef=1.0, tokens=4, ld=8, mask=None, counts=P, live=P,
                            d_loss=P, d_logits=P, ld_d=8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(topk=0), 1), (dict(experts=2000, ld=2000), 1), (dict(logits=None), 1), (dict(counts=None), 1),
    (dict(live=None), 1), (dict(type=3), 2), (dict(ld=7), 3), (dict(logits=P + 1), 4), (dict(live=P + 2), 4),
])
def test_balance_refusals(change, status):
    assert R.lib().balance_loss(ctypes.byref(loss(**change)), None) == status
    assert R.lib().balance_grad(ctypes.byref(grad(**change)), None) == status


def test_balance_own_refusals():
    for change, status in ((dict(loss=None), 1), (dict(prob=None), 1), (dict(workspace=None), 1), (dict(workspace=P + 8), 4)):
        assert R.lib().balance_loss(ctypes.byref(loss(**change)), None) == status
    for change, status in ((dict(d_loss=None), 1), (dict(d_logits=None), 1), (dict(ld_d=7), 3), (dict(d_logits=P + 1), 4)):
        assert R.lib().balance_grad(ctypes.byref(grad(**change)), None) == status
    assert R.lib().balance_loss(None, None) == 1
    assert R.lib().balance_grad(None, None) == 1
    assert R.lib().balance_grad(ctypes.byref(grad(tokens=0, logits=None, d_logits=None)), None) == 0


def test_workspace_sizes():
    assert R.workspace_size(0, 1, 1) > 0
    assert R.workspace_size(16384, 8, 256) >= 64 * 256 * 4
    for args in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 4, 8)):
        with pytest.raises(H.GemmError) as err:
            R.workspace_size(*args)
        assert err.value.status == 1


def test_shapes_that_do_not_fit():
    """The binding's own checks, on host tensors: nothing reaches the library."""
    import torch
    x = torch.zeros(4, 256)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    bad = [dict(q=q[:, :255], scale=s), dict(q=q, scale=s[:, :1]), dict(q=q, scale=s.double()), dict(q=q.t(), scale=s),
           dict(q=q, scale=s, row_index=torch.zeros(3, dtype=torch.int32)), dict(q=q, scale=s, row_index=torch.zeros(4)),
           dict(q=x, scale=s), dict(qt=q, scale_t=s)]
    for kw in bad:
        with pytest.raises(H.GemmError):
            S.quantize(x, stream=0, **kw)
    wide = torch.zeros(256).expand(4, 256)    # rows that overlap: a row stride of 0
    for x2, kw in ((wide, dict(q=q, scale=s)), (x, dict(q=torch.zeros(256, dtype=torch.uint8).expand(4, 256), scale=s)),
                   (x.t(), dict(q=torch.zeros(256, 4, dtype=torch.uint8), scale=torch.zeros(256, 1)))):
        with pytest.raises(H.GemmError):
            S.quantize(x2, stream=0, **kw)
    i = dict(dtype=torch.int32)
    counts, live, one = torch.zeros(8, **i), torch.zeros(1, **i), torch.zeros(1)
    ws = torch.zeros(1 << 14, dtype=torch.uint8)
    with pytest.raises(H.GemmError):
        R.balance_loss(torch.zeros(8).expand(4, 8), counts, 2, one, torch.zeros(8), live, workspace=ws, stream=0)
    for x2, d in ((torch.zeros(8).expand(4, 8), torch.zeros(4, 8)), (torch.zeros(4, 8), torch.zeros(8).expand(4, 8)),
                  (torch.zeros(4, 8), torch.zeros(4, 8).double())):
        with pytest.raises(H.GemmError):
            R.balance_grad(x2, counts, 2, live, one, d, stream=0)
    ok = dict(ids=torch.zeros(4, 2, **i), counts=torch.zeros(8, **i), offsets=torch.zeros(9, **i),
              workspace=torch.zeros(1 << 14, dtype=torch.uint8))
    for kw in (dict(ids=torch.zeros(4, 2)), dict(ids=torch.zeros(2, **i).expand(4, 2)),
               dict(offsets=torch.zeros(8, **i)), dict(counts=torch.zeros(8)),
               dict(slot=torch.zeros(4, 1, **i)), dict(mask=torch.zeros(3, dtype=torch.uint8)), dict(workspace=None),
               dict(workspace=torch.zeros(1, dtype=torch.uint8)), dict(mask=torch.zeros(4))):
        with pytest.raises(H.GemmError):
            R.route(**{**ok, **kw}, stream=0)
