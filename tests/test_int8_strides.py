"""Tensors of an int8 product whose strides are not the description's: the binding refuses them, as the
library would read other values, and takes every layout that it reads right (on the host; the library's
call is replaced)."""
import types

import pytest
import torch

from hierarchical_tiling_amd import htgemm as H
from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htscaled as S

I8, I32, BF16 = (dict(dtype=t) for t in (torch.int8, torch.int32, torch.bfloat16))


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: -1)


@pytest.fixture()
def taken(monkeypatch):
    """The arguments of the library's calls, of which none is made."""
    calls = []
    real = Q.lib()
    monkeypatch.setattr(Q, "_lib", types.SimpleNamespace(
        **{n: getattr(real, n) for n in Q.EXPORTED if n != "gemm_int8_run"},
        gemm_int8_run=lambda *a: calls.append(Q._ARGS.unpack(a[1])) or 0))
    return calls


M, N, K = 6, 5, 16


def product(**kw):
    return Q.Int8Gemm(Q.make_desc(M, N, K, **{**dict(lda=32, ldb=16, ldd=8, ldc=5, bias=True), **kw}))


def tensors():
    return dict(A=torch.zeros(M, 32, **I8)[:, :K], a_scale=torch.zeros(M), B=torch.zeros(N, K, **I8), b_scale=torch.zeros(N),
                D=torch.zeros(M, 8, **BF16)[:, :N], C=torch.zeros(M, N, **BF16), bias=torch.zeros(N, **BF16), beta=1.0)


@pytest.mark.parametrize("name,bad", [
    ("a_scale", torch.zeros(2 * M)[::2]), ("a_scale", torch.zeros(M, 4)[:, :1]), ("a_scale", torch.zeros(M, 4)[:, 0]),
    ("b_scale", torch.zeros(N, 2)[:, 1]), ("bias", torch.zeros(N, 2, **BF16)[:, 0]), ("A", torch.zeros(M, 48, **I8)[:, :K]),
    ("A", torch.zeros(M + 6, K, **I8)[:M]), ("A", torch.zeros(32, M, **I8).t()[:, :K]), ("B", torch.zeros(N, 32, **I8)[:, :K]),
    ("D", torch.zeros(M, 16, **BF16)[:, :N]), ("D", torch.zeros(100, **BF16)[: M * N].view(M, N)),
    ("C", torch.zeros(M, 8, **BF16)[:, :N]), ("C", torch.zeros(N, M + 5, **BF16).t()[:M])])
def test_refused(name, bad, taken):
    h, good = product(), tensors()
    h.run(**good)
    with pytest.raises(H.GemmError) as e:
        h.run(**{**good, name: bad})
    assert e.value.status == H.GEMM_ERR_INVALID_ARG and len(taken) == 1


def test_offsets_that_are_not_neighbours(taken):
    h = product(groups="rows", batch=2, b_stride_l=N * K, b_scale_l=N, ldd=N, bias=False)
    good = dict(A=torch.zeros(M, 32, **I8)[:, :K], a_scale=torch.zeros(M), B=torch.zeros(2, N, K, **I8), b_scale=torch.zeros(2, N),
                D=torch.zeros(M, N, **BF16), offsets=torch.zeros(3, **I32))
    h.run(**good)
    with pytest.raises(H.GemmError):
        h.run(**{**good, "offsets": torch.zeros(6, **I32)[::2]})
    assert len(taken) == 1


def test_layouts_that_are_taken(taken):
    """Flat memory, more dimensions, scales with a dimension of one, groups' scales rows apart, addresses."""
    h, good = product(), tensors()
    flat = torch.zeros(M * 32, **I8)
    for name, other in (("A", flat), ("A", flat.data_ptr()), ("A", torch.zeros(1, M, 32, **I8)[:, :, :K]), ("B", torch.zeros(N, 1, K, **I8)),
                        ("a_scale", torch.zeros(M, 1)), ("a_scale", torch.zeros(1, 2 * M)[:, 2: M + 2]),
                        ("b_scale", torch.zeros(3 * N)[N: 2 * N]), ("D", torch.zeros(M * 8, **BF16)),
                        ("bias", torch.zeros(1, N, **BF16)), ("C", torch.zeros(M + 1, N, **BF16)[1:])):
        h.run(**{**good, name: other})
    h = product(groups="rows", batch=3, b_stride_l=8 * 32, ldb=32, b_scale_l=8, ldd=N, ldc=0, bias=False)
    h.run(good["A"], good["a_scale"], torch.zeros(3, 8, 32, **I8)[:, :N, :K], torch.zeros(3, 8)[:, :N], torch.zeros(M, N, **BF16),
          offsets=torch.zeros(4, **I32))
    h = Q.Int8Gemm(Q.make_desc(1, 1, 1, lda=7, ldb=9, ldd=3))
    h.run(torch.zeros(1, 7, **I8)[:, :1], torch.zeros(4)[::4], torch.zeros(1, 9, **I8)[:, 3:4], torch.zeros(2)[1:],
          torch.zeros(5, 2, **BF16)[2:3, 1:])
    assert len(taken) == 12
