"""Operands and outputs of more than 2^31 and 2^32 values, at their ends.  Whole codes and scales that
are powers of two: the products are exact."""
import pytest
import torch

from hierarchical_tiling_amd import htscaled as S
from scaled_util import BLOCK, up

pytestmark = pytest.mark.gpu


def whole(g, rows, K, ld=None):
    """Codes of whole numbers from -3 to 3, rows of a pitch ld; the pitch's bytes are NaN codes."""
    ld = ld or K
    q = torch.full((rows, ld), 0x7f, dtype=torch.uint8, device="cuda")
    table = torch.arange(-3, 4, device="cuda").float().to(torch.float8_e4m3fn).view(torch.uint8)
    step = max(1, (1 << 27) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q[r:r + n, :K] = table[torch.randint(0, 7, (n, K), generator=g, device="cuda", dtype=torch.uint8).int()]
    return q


def values(q, K):
    return q[:, :K].contiguous().view(torch.float8_e4m3fn).float().double()


def scales(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


def want(a, sa, b, sb, K):
    """sa (rows, blocks), sb (blocks of 128 rows of b, blocks)."""
    va = values(a, K) * sa.double().repeat_interleave(BLOCK, 1)[:, :K]
    vb = values(b, K) * sb.double().repeat_interleave(BLOCK, 0)[:b.shape[0]].repeat_interleave(BLOCK, 1)[:, :K]
    return torch.mm(va, vb.t().contiguous())


@pytest.mark.parametrize("M,N,K,lda,ldd,out", [
    (300_001, 72, 8192, 8192, 72, "f32"),           # A of 2.5 GB
    (300_001, 520, 8192, 8192, 520, "bf16"),
    (700, 300, 272, 4_000_000, 300, "bf16"),        # rows of A far apart
    (40, 130, 1040, 7_000_000, 130, "f32"),
    (263_000, 16_400, 128, 128, 16_400, "bf16"),    # D of 4.3 G values
    (1_030, 272, 144, 144, 4_200_000, "f32"),
    (33, 70, 400, 9_000_000, 70, "bf16")])          # too far for the 16-byte loads' offsets
def test_products(M, N, K, lda, ldd, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    a, b, kb = whole(g, M, K, lda), whole(g, N, K), up(K, BLOCK)
    sa, sb = scales(g, kb, M), scales(g, up(N, BLOCK), kb)
    h = S.ScaledGemm(S.make_desc(M, N, K, out, lda=lda, ldb=K, ldd=ldd, a_scale_strides=(1, M), b_scale_strides=(kb, 1)))
    d = torch.full((M, ldd), -7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    h.run(a, sa, b, sb, d, workspace=torch.empty(max(1, h.workspace_bytes), dtype=torch.uint8, device="cuda"))
    for rows in (slice(0, 400), slice(M // 2, M // 2 + 300), slice(max(0, M - 700), M)):
        got = d[rows, :N]
        assert torch.equal(got, want(a[rows], sa[:, rows].t(), b, sb, K).to(got.dtype))
    if ldd > N:
        assert (d[-1, N:] == -7.0).all() and (d[0, N:] == -7.0).all()


@pytest.mark.parametrize("E,N,K,rows", [(70, 4100, 8192, 200), (9, 30_000, 8192, 2_500)])
def test_experts_with_many_weights(E, N, K, rows):
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    kb, nb = K // BLOCK, up(N, BLOCK)
    a, b = whole(g, rows, K), whole(g, E * N, K)
    sa, sb = scales(g, kb, rows), scales(g, E, nb, kb)
    offsets = torch.tensor([rows * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    h = S.ScaledGemm(S.make_desc(rows, N, K, lda=K, ldb=K, ldd=N, a_scale_strides=(1, rows), b_scale_strides=(kb, 1),
                                 groups="rows", batch=E, b_stride_l=N * K, b_scale_l=nb * kb))
    d = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    h.run(a, sa, b, sb, d, offsets=offsets)
    for e in (0, E // 2, E - 1):
        r = slice(rows * e // E, rows * (e + 1) // E)
        assert torch.equal(d[r], want(a[r], sa[:, r].t(), b[e * N:(e + 1) * N], sb[e], K).to(torch.bfloat16))


def test_experts_gradients_of_more_than_32_bits():
    E, M, N, rows = 40, 9_000, 12_000, 40 * 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    a, b, kb = whole(g, M, rows), whole(g, N, rows), rows // BLOCK
    sa, sb = scales(g, kb, M), scales(g, kb, N)
    offsets = torch.arange(0, rows + 1, BLOCK, dtype=torch.int32, device="cuda")
    h = S.ScaledGemm(S.make_desc(M, N, rows, lda=rows, ldb=rows, ldd=N, b_block=1, a_scale_strides=(1, M), b_scale_strides=(1, N),
                                 groups="k", batch=E, d_stride_l=M * N))
    d = torch.empty(E, M, N, dtype=torch.bfloat16, device="cuda")
    h.run(a, sa, b, sb, d, offsets=offsets)
    for e in (0, 20, 39):
        s = slice(e * BLOCK, (e + 1) * BLOCK)
        x = values(a[:, s], BLOCK) * sa[e].double()[:, None]
        y = values(b[:, s], BLOCK) * sb[e].double()[:, None]
        assert torch.equal(d[e], torch.mm(x, y.t().contiguous()).to(torch.bfloat16))


@pytest.mark.parametrize("rows,cols,both", [(1_050_000, 4_100, False), (600_000, 8_200, True), (5, 900_000_000, True)])
def test_quantise(rows, cols, both):
    """Of more than 2^32 values; the ends by themselves give the same codes and scales."""
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 30):
        flat[i:i + (1 << 30)].normal_(generator=g)
    q, s = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(up(cols, BLOCK), rows, device="cuda").t()
    qt = torch.empty(cols, rows, dtype=torch.uint8, device="cuda") if both else None
    st = torch.empty(up(rows, BLOCK), cols, device="cuda").t() if both else None
    S.quantize(x, q, s, qt, st)
    r0, c0 = max(0, rows - 1) // BLOCK * BLOCK, max(0, cols - 1) // BLOCK * BLOCK
    for r, c in ((slice(r0, rows), slice(c0, cols)), (slice(0, min(rows, BLOCK)), slice(c0, cols)), (slice(r0, rows), slice(0, BLOCK))):
        part = x[r, c].contiguous()
        n, m = part.shape
        q1, s1 = torch.empty(n, m, dtype=torch.uint8, device="cuda"), torch.empty(n, 1, device="cuda")
        qt1, st1 = torch.empty(m, n, dtype=torch.uint8, device="cuda"), torch.empty(m, 1, device="cuda")
        S.quantize(part, q1, s1, qt1, st1)
        assert torch.equal(q[r, c], q1) and torch.equal(s[r, c.start // BLOCK], s1[:, 0])
        if both:
            assert torch.equal(qt[c, r], qt1) and torch.equal(st[c, r.start // BLOCK], st1[:, 0])
