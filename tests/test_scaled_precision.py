"""What include/htscaled.h promises of the sums: for a bf16 D within 2^-10 of the sum of the sizes of
what is added, for an fp32 D fp32's own accuracy, also where large products cancel."""
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from scaled_util import BLOCK, codes, spread_scales, up, values

pytestmark = pytest.mark.gpu

OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def run(a, sa, b, sb, out, **kw):
    M, K = a.shape
    N = b.shape[0]
    h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=K, ldb=K, ldd=N, a_scale_strides=sa.stride(), b_scale_strides=sb.stride(), **kw))
    d = torch.empty(M, N, dtype=OUT[out], device="cuda")
    h.run(a, sa, b, sb, d, workspace=torch.empty(max(1, h.workspace_bytes), dtype=torch.uint8, device="cuda"))
    return d, h.info.name.decode()


def check(a, sa, b, sb, out, **kw):
    """The bounds: of an 8-bit group of 8 products each but the largest loses less than 2^-13 of the
    largest, so 7 * 2^-13 < 2^-10 of the group's sizes; the fp32 additions, of 16 groups and of the
    blocks and 8 steps behind them, at most an ulp, 2^-23, of all the sizes; the rounding of D, half
    a step.  With an fp32 D 128 additions in place of the groups, half an ulp each, and no first part."""
    M, K = a.shape
    va, vb = values(a) * spread_scales(sa, M, K, 1), values(b) * spread_scales(sb, b.shape[0], K, BLOCK)
    y, size = torch.mm(va, vb.t().contiguous()), torch.mm(va.abs(), vb.abs().t().contiguous())
    d, name = run(a, sa, b, sb, out, **kw)
    blocks = up(K, BLOCK)
    tol = size * (2.0 ** -10 + (16 + blocks + 8) * 2.0 ** -23) + y.abs() * 2.0 ** -8 if out == "bf16" else \
        size * ((128 + blocks + 8) * 2.0 ** -24) + y.abs() * 2.0 ** -24
    bad = (d.double() - y).abs() > tol
    assert not bad.any(), (name, int(bad.sum()), float(((d.double() - y).abs() / size).max()))
    return d, y, size


def outliers(g, rows, K):
    """Codes of small values with a large one here and there, in pairs that may cancel."""
    v = torch.randn(rows, K, generator=g, device="cuda") * 2
    at = torch.rand(rows, K, generator=g, device="cuda") < 2.0 / BLOCK
    return torch.where(at, v.sign() * 448, v).to(torch.float8_e4m3fn).view(torch.uint8)


SHAPES = [(16, 16, 128), (5, 300, 100), (16, 4096, 2048), (64, 4096, 1024), (333, 2048, 1040), (600, 4096, 512), (4096, 4096, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_outliers(M, N, K, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    a, b = outliers(g, M, K), outliers(g, N, K)
    kb = up(K, BLOCK)
    sa = torch.exp(torch.randn(M, kb, generator=g, device="cuda"))
    sb = torch.exp(torch.randn(up(N, BLOCK), kb, generator=g, device="cuda"))
    check(a, sa.t().contiguous().t(), b, sb, out)


def spread_of_exponents(g, rows, K):
    """Codes of all exponents alike: most of a group lies far below its largest."""
    e = torch.randint(-9, 9, (rows, K), generator=g, device="cuda")
    m = 1 + torch.randint(0, 8, (rows, K), generator=g, device="cuda") / 8
    s = torch.randint(0, 2, (rows, K), generator=g, device="cuda") * 2 - 1
    return torch.ldexp(s * m, e).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_all_exponents(M, N, K, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    kb = up(K, BLOCK)
    one = torch.ones(up(max(M, N), 1), kb, device="cuda")
    check(spread_of_exponents(g, M, K), one[:M].t().contiguous().t(), spread_of_exponents(g, N, K), one[:up(N, BLOCK)], out)


@pytest.mark.parametrize("small", [1.0, 2.0, 3.75, 7.0, 7.5, 8.0, 15.0])
def test_small_products_beside_large_ones_that_cancel(small):
    """256 * 256 and -256 * 256 in two groups of 8, each among 7 small products: a bf16 D may lose
    those whole (7 of 7.0 are more than 2^-11 of the sizes), an fp32 D has them exactly."""
    K = 128
    v = torch.zeros(16, K, device="cuda")
    w = torch.zeros(16, K, device="cuda")
    for i in range(16):
        p, q = 8 * i, 8 * ((i + 5) % 16)
        v[i, p:p + 8], v[i, q:q + 8], w[i, p:p + 8], w[i, q:q + 8] = small, small, 1, 1
        v[i, p + i % 8], w[i, p + i % 8] = 256, 256
        v[i, q + (3 * i) % 8], w[i, q + (3 * i) % 8] = -256, 256
    a, b = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (v, w))
    one = torch.ones(16, 1, device="cuda")
    check(a, one, b, one[:1], "bf16")
    d, y, _ = check(a, one, b, one[:1], "f32")
    assert (d.diagonal() == 14 * small).all() and torch.equal(d.double(), y)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_long_sum_of_both_signs(out):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    M, N, K = 40, 130, 65536
    kb = K // BLOCK
    check(codes(g, M, K), torch.ones(M, kb, device="cuda"), codes(g, N, K), torch.ones(2, kb, device="cuda"), out)
