"""Calls of the operators in 8-bit integers and of the rows of a routing that have nothing to do, with the
empty tensors (whose address is 0) that a program has for them, on the host."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from hierarchical_tiling_amd import htroute as R
from hierarchical_tiling_amd import htscaled as S


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    """The device check finds a gfx950, and the current device is the tensors'."""
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(S, "_device", lambda: -1)


@pytest.mark.parametrize("M,N", [(0, 5), (5, 0), (0, 0)])
@pytest.mark.parametrize("K", [0, 16])
def test_product_of_no_rows_or_columns(M, N, K):
    h = Q.Int8Gemm(Q.make_desc(M, N, K, "f32", lda=K, ldb=K, ldd=N, ldc=N + 1, bias=True))
    a, b = torch.empty(M, K, dtype=torch.int8), torch.empty(N, K, dtype=torch.int8)
    h.run(a, torch.empty(M), b, torch.empty(N), torch.empty(M, N), C=torch.empty(M, N), bias=torch.empty(N), beta=1.0)


@pytest.mark.parametrize("T,n,H", [(0, 5, 0), (4, 0, 8), (4, 5, 0), (0, 0, 8), (0, 0, 0)])
def test_rows_of_nothing(T, n, H):
    """Without columns, or without rows and tokens to write; gradients that are asked for one by one."""
    x, y, order, slot = torch.empty(T, H), torch.empty(n, H), torch.zeros(n, dtype=torch.int32), torch.zeros(T, 2, dtype=torch.int32)
    w = torch.empty(T, 2)
    R.gather(x, order, slot, y)
    if T == 0 or H == 0:
        R.combine(y, slot, x, weights=w, add=torch.empty(T, H))
    R.combine_grad(x, None, order, slot, w, torch.empty(n, H), None)
    if T == 0:
        R.combine_grad(x, y, order, slot, w, None, torch.empty(T, 2))
        R.combine_grad(x, y, order, slot, w, torch.empty(n, H), torch.empty(T, 2))
