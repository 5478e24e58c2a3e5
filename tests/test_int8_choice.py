"""Which kernel the sizes of test_int8_epilogue.py are for, asked on the host."""
import pytest

from hierarchical_tiling_amd import htint8 as Q
from test_int8_epilogue import BATCHES, GROUPS, KERNELS, WITHOUT_K, pitch_of

TYPES = ["bf16", "f16", "f32"]


@pytest.fixture(autouse=True)
def fake_gfx950(monkeypatch):
    monkeypatch.setenv("HTGEMM_FAKE_ARCH", "gfx950")


def name(M, N, K, out, ld, **kw):
    return Q.Int8Gemm(Q.make_desc(M, N, K, out, lda=ld, ldb=ld, ldd=N, **kw)).info.name.decode()


@pytest.mark.parametrize("out", TYPES)
def test_kernels_of_the_epilogue_tests(out):
    for kernel, M, N, K, on16 in KERNELS:
        assert name(M, N, K, out, pitch_of(K, on16), split_k=1) == kernel
    for kernel, M, N, ld in WITHOUT_K:
        assert name(M, N, 0, out, ld) == kernel
    for kernel, M, N, K, batch in BATCHES:
        P = pitch_of(K, True)
        assert name(M, N, K, out, P, batch=batch, a_stride_l=M * P, b_stride_l=N * P, d_stride_l=M * N) == kernel
    for kernel, N, K, on16, sizes in GROUPS:
        P = pitch_of(K, on16)
        assert name(sum(sizes) + 14, N, K, out, P, groups="rows", batch=len(sizes), b_stride_l=N * P) == kernel


def test_every_kernel_with_an_epilogue_of_its_own_is_tested():
    assert {k for k, *_ in KERNELS} == {"any_64x128", "any_128x128", "tile_64x128_w2x2", "tile_64x128_w2x2x2",
                                        "tile_128x128_w2x2", "tile_128x128_w2x2x2", "pingpong_256x256"}
