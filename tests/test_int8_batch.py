"""The batch form of int8 products at strides of every kind: rows at any byte, operands that products share,
outputs that lie between each other, the most products."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import TYPE, codes, gen, reference, scales
from test_int8_epilogue import near, normal

pytestmark = pytest.mark.gpu


def handle(M, N, K, out, **kw):
    h = Q.Int8Gemm(Q.make_desc(M, N, K, out, **kw))
    return h, torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,batch,kernel", [(300, 200, 150, 3, "any_64x128"), (1030, 520, 130, 9, "any_128x128"), (5, 7, 3, 40, "any_64x128"),
                                                (257, 260, 300, 12, "any")])
def test_rows_at_any_byte(M, N, K, batch, kernel, out):
    """Odd leading dimensions, and products an odd number of bytes apart."""
    g = gen(M)
    a_l, b_l = M * (K + 1) + 5, N * (K + 3) + 2
    a, b = (torch.randint(-128, 128, (batch * n,), generator=g, device="cuda", dtype=torch.int8) for n in (a_l, b_l))
    sa, sb = scales(g, batch * (M + 1)).view(batch, M + 1)[:, :M], scales(g, batch * N).view(batch, N)
    c, bias, d = normal(g, out, batch, M, N), normal(g, out, N), torch.empty(batch, M, N, dtype=TYPE[out], device="cuda")
    h, ws = handle(M, N, K, out, lda=K + 1, ldb=K + 3, ldd=N, ldc=N, bias=True, act="relu", batch=batch, a_stride_l=a_l,
                   b_stride_l=b_l, c_stride_l=M * N, d_stride_l=M * N, a_scale_l=M + 1, b_scale_l=N)
    assert h.info.name.startswith(kernel.encode())
    h.run(a, sa, b, sb, d, C=c, bias=bias, beta=0.5, workspace=ws)
    for i in range(batch):
        ai, bi = a[i * a_l:].as_strided((M, K), (K + 1, 1)), b[i * b_l:].as_strided((N, K), (K + 3, 1))
        near(d[i], *reference(ai, sa[i], bi, sb[i], out, 1.0, 0.5, c[i], bias, "relu"))


@pytest.mark.parametrize("M,N,K", [(20, 64, 160), (300, 256, 160), (700, 520, 160)])
def test_one_a_for_all_and_outputs_side_by_side(M, N, K):
    """A and its scales shared; D's rows hold the products one after the other."""
    g = gen(N)
    batch = 3
    a, b, sa, sb = codes(g, M, K), codes(g, batch * N, K), scales(g, M), scales(g, batch * N)
    d = torch.empty(M, batch * N, device="cuda")
    h, ws = handle(M, N, K, "f32", lda=K, ldb=K, ldd=batch * N, batch=batch, b_stride_l=N * K, d_stride_l=N, b_scale_l=N)
    h.run(a, sa, b, sb, d, workspace=ws)
    near(d, *reference(a, sa, b, sb, "f32"))


@pytest.mark.parametrize("lda", [16, 5])
def test_most_products(lda):
    g = gen(lda)
    batch, M, N, K = 65535, 2, 3, 5
    a, b, sa, sb = codes(g, batch * M, K, lda), codes(g, N, K, 16), scales(g, batch * M), scales(g, N)
    d = torch.full((batch * M + 1, N), -7.0, device="cuda")
    h, ws = handle(M, N, K, "f32", lda=lda, ldb=16, ldd=N, batch=batch, a_stride_l=M * lda, d_stride_l=M * N, a_scale_l=M)
    h.run(a, sa, b, sb, d, workspace=ws)
    near(d[:-1], *reference(a, sa, b, sb, "f32"))
    assert (d[-1] == -7.0).all()
