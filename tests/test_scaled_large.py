"""Sizes whose launch would have 2^32 threads or more, which the runtime would run as what is left
modulo 2^32."""
import ctypes

import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from hierarchical_tiling_amd.htgemm import GEMM_ERR_INVALID_ARG, GemmError


@pytest.mark.gpu
def test_quantise_more_rows_than_a_launch_has_waves():
    """2^26 rows are 2^26 waves of 64; the halves by themselves give the same bits."""
    rows, half = 2 ** 26 + 3, 2 ** 25
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(rows, 1, generator=g, device="cuda").to(torch.float16)
    q, s = torch.full((rows, 1), 0xee, dtype=torch.uint8, device="cuda"), torch.full((rows, 1), -1.0, device="cuda")
    S.quantize(x, q, s)
    for part in (slice(0, half), slice(half, rows)):
        q1, s1 = torch.empty_like(q[part]), torch.empty_like(s[part])
        S.quantize(x[part], q1, s1)
        assert torch.equal(q[part], q1) and torch.equal(s[part], s1)
    live = x != 0
    assert ((q & 0x7f == 0x7e) == live).all()    # the largest code, each row's only value
    # scale = t / 448 and 448 * scale, an ulp at most each
    assert ((s * 448 - x.float().abs()).abs()[live] <= 2.0 ** -22 * x.float().abs()[live]).all()


@pytest.mark.parametrize("sizes", [
    dict(M=2 ** 30 - 1, N=64, K=1), dict(M=64, N=2 ** 30 - 1, K=3), dict(M=2 ** 30 - 1, N=128, K=16), dict(M=16, N=2 ** 29, K=16),
    dict(M=5, N=2 ** 30 - 1, K=128), dict(M=2 ** 20, N=2 ** 20, K=256), dict(M=2 ** 24, N=2 ** 24, K=256),
    dict(M=2 ** 30 - 1, N=2 ** 30 - 1, K=128), dict(M=2 ** 30 - 1, N=2 ** 30 - 1, K=1), dict(M=100, N=2 ** 29, K=128, out="f32"),
    dict(M=2 ** 30 - 1, N=200, K=128, groups="rows", batch=65535), dict(M=300, N=2 ** 30 - 1, K=64, groups="k", batch=9, d_stride_l=1)])
def test_products_that_no_launch_holds(sizes, monkeypatch):
    """A handle's launch has fewer than 2^32 threads along x, or there is no handle."""
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    N, K = sizes["N"], sizes["K"]
    try:
        h = S.ScaledGemm(S.make_desc(**{**dict(lda=K, ldb=K, ldd=N, a_scale_strides=(1, sizes["M"]), b_scale_strides=(1, 1)),
                                        **sizes}))
    except GemmError as e:
        assert e.status == GEMM_ERR_INVALID_ARG
        assert sizes["M"] * N > 2 ** 35     # of 64 x 64 tiles, 256 threads each, 2^36 outputs fit
        return
    i = h.info
    along_x = i.grid // (i.split_k * (sizes["batch"] if sizes.get("groups") == "k" else 1))
    assert along_x * i.waves * 64 < 2 ** 32


def test_misaligned_products_that_no_launch_holds(monkeypatch):
    """Operands that only the single-byte loads can read take smaller tiles than the handle chose for."""
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")
    M, N, K = 64, 2 ** 30 - 1, 16
    h = S.ScaledGemm(S.make_desc(M, N, K, lda=K, ldb=K, ldd=N, a_scale_strides=(1, M), b_scale_strides=(1, 1), split_k=1))
    assert h.info.bn > 64
    a = 1 << 20
    args = S.gemm_scaled_args(A=a + 1, a_scale=a, B=a, b_scale=a, D=a)
    assert S.lib().gemm_scaled_run(h.handle, ctypes.byref(args), None) == GEMM_ERR_INVALID_ARG
