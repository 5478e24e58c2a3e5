"""A product's bits go by its operands alone: not by the slices of k, the kernel, the alignment of the
operands, or how many rows there are beside a row, with alpha, C, bias and activations."""
import pytest
import torch

from hierarchical_tiling_amd import htint8 as Q
from int8_util import I32, TYPE, codes, gen, scales

pytestmark = pytest.mark.gpu


class Product:
    def __init__(self, M, N, K, out):
        g = gen(M + N + K)
        self.M, self.N, self.K, self.out, self.P = M, N, K, out, -(-K // 16) * 16
        self.a, self.b, self.sa, self.sb = codes(g, M, K, self.P), codes(g, N, K, self.P), scales(g, M), scales(g, N)
        self.c = torch.randn(M, N, generator=g, device="cuda").to(TYPE[out])
        self.bias = torch.randn(N, generator=g, device="cuda").to(TYPE[out])

    def run(self, rows, beta, bias, act, split_k=0, odd=False, groups=False):
        """The first `rows` rows; odd: from operands whose rows lie off 16 bytes.  (D, kernel)"""
        P = self.P + 1 if odd else self.P
        a, b = self.a[:rows], self.b
        if odd:
            a, b = (torch.nn.functional.pad(t, (0, P - self.K)) for t in (a, b))
        kw = dict(groups="rows", batch=1, b_stride_l=0, b_scale_l=0) if groups else {}
        h = Q.Int8Gemm(Q.make_desc(rows, self.N, self.K, self.out, lda=P, ldb=P, ldd=self.N, ldc=self.N, bias=bias, act=act,
                                   split_k=split_k, **kw))
        d = torch.empty(rows, self.N, dtype=TYPE[self.out], device="cuda")
        ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
        h.run(a, self.sa[:rows], b, self.sb, d, C=self.c, bias=self.bias if bias else None, alpha=0.7, beta=beta, workspace=ws,
              offsets=torch.tensor([0, rows], **I32) if groups else None)
        return d, h.info.name.decode()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(333, 1024, 600), (333, 1003, 600), (333, 4096, 4100), (2048, 2100, 530), (2300, 4099, 1030)])
def test_same_bits(M, N, K, out):
    p = Product(M, N, K, out)
    for beta, bias, act in ((0.0, False, "none"), (0.0, True, "none"), (1.3, False, "none"), (1.3, True, "none"), (1.3, True, "silu"),
                            (0.0, True, "gelu"), (1.3, True, "relu")):
        want, name = p.run(M, beta, bias, act, split_k=1)
        kernels = {name}
        for kw in (dict(split_k=2), dict(split_k=3), dict(split_k=1, odd=True), dict(split_k=2, odd=True), dict(groups=True)):
            got, name = p.run(M, beta, bias, act, **kw)
            kernels.add(name)
            assert torch.equal(got, want), (beta, bias, act, kw, name, int((got != want).sum()))
        for rows in (1, 16, 40, 64, 130):
            for split_k in (1, 2):
                got, name = p.run(rows, beta, bias, act, split_k=split_k)
                kernels.add(name)
                assert torch.equal(got, want[:rows]), (beta, bias, act, rows, split_k, name, int((got != want[:rows]).sum()))
        assert len(kernels) >= 4, kernels
